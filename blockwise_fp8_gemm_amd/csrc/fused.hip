// Operators on either side of the blockwise-FP8 GEMMs whose results are GEMM
// operands, quantised where they are formed (gfx950).
//
//   norm          z = BF16(x + residual), r = 1 / sqrt(mean z^2 + eps),
//                 n = z r w                    -> the q/k/v and gate/up operand
//   norm gradient dx = dres + r (g - xh mean(g xh)), g = w dy, xh = z r
//                                              -> dY of the linear before
//                 dw = sum over tokens of dy xh
//   activation    du = dh silu(g), dg = dh u silu'(g)
//   gradient                                   -> dY of the gate/up product
//
// The feed-forward and norms are those of the Qwen3-1.7B configuration that
// the Puro-2B-Base model card's configuration table names; the card keeps
// norms in BF16 / FP32 and the GEMMs that read them in blockwise E4M3.
//
// Values are formed in FP32 and quantised unrounded: a block's scale is
// amax / 448 (or the power-of-two rule) of the FP32 values and a code is
// E4M3(v / s).  Rounding to BF16 first would only add an error, and would
// let a last-bit difference of a sum move a scale by 2^-8.
//
// All of them are HBM-bound.  The token blocks of one column span 128 tokens
// and the norm's statistics a whole row, so the norm and its gradient take
// two passes: per-row statistics, then 128 x 128 tiles that hold one block of
// each kind per token and per column.
#include "common.h"
#include "kernels.h"

namespace puro {

namespace {

constexpr int TT = 512;   // threads of a tile kernel: 16 column groups x 32 token groups

template <int CTRL> __device__ __forceinline__ float dpp_f(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}

// Max over each row of 16 lanes (DPP row rotates; every lane ends with it).
__device__ __forceinline__ float max16(float v)
{
    v = fmaxf(v, dpp_f<0x128>(v));
    v = fmaxf(v, dpp_f<0x124>(v));
    v = fmaxf(v, dpp_f<0x122>(v));
    return fmaxf(v, dpp_f<0x121>(v));
}

// Sum over the wave (every lane ends with it).
__device__ __forceinline__ float sum64(float v)
{
    v += dpp_f<0x128>(v);
    v += dpp_f<0x124>(v);
    v += dpp_f<0x122>(v);
    v += dpp_f<0x121>(v);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// Code factor of a block: v * r rounds within 2 ulps of v / s.  r is 0 for a
// zero scale (codes +-0 by sign); a subnormal scale (1 / s could overflow)
// divides instead, which SLOW selects for a whole tile or row run.
__device__ __forceinline__ float scale_inv(float s) { return s >= 0x1p-126f ? 1.0f / s : 0.0f; }
__device__ __forceinline__ bool scale_slow(float s) { return s != 0.0f && s < 0x1p-126f; }

template <bool SLOW> __device__ __forceinline__ float code_arg(float v, float s, float r)
{
    if (SLOW && scale_slow(s))
        return v / s;
    return v * r;
}

template <bool SLOW>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float s, float r)
{
    return e4m3x4(code_arg<SLOW>(a, s, r), code_arg<SLOW>(b, s, r), code_arg<SLOW>(c, s, r), code_arg<SLOW>(d, s, r));
}

// Eight BF16 values of a row from column c0 on, zeros at and past cols.
__device__ __forceinline__ uint4 load8_bf16(const uint16_t *row, int64_t c0, int64_t cols)
{
    if (c0 + 8 <= cols)
        return *reinterpret_cast<const uint4 *>(row + c0);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (c0 + j < cols)
            w[j >> 1] |= (uint32_t)row[c0 + j] << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8_bf16(uint16_t *row, int64_t c0, int64_t cols, const uint32_t w[4])
{
    if (c0 + 8 <= cols) {
        store_nt(row + c0, w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (c0 + j < cols)
            row[c0 + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
}

__device__ __forceinline__ void store8_codes(uint8_t *row, int64_t c0, int64_t cols, uint32_t lo, uint32_t hi)
{
    if (c0 + 8 <= cols) {
        store_nt(row + c0, lo, hi);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (c0 + j < cols)
            row[c0 + j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
}

__device__ __forceinline__ void unpack8(const uint4 &a, float v[8])
{
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
}

// Eight norm weights from column c0 on (zeros past cols).
__device__ __forceinline__ void load8_weight(const void *w, int wbf16, int64_t c0, int64_t cols, float v[8])
{
    if (wbf16) {
        unpack8(load8_bf16((const uint16_t *)w, c0, cols), v);
        return;
    }
    const float *p = (const float *)w;
    if (c0 + 8 <= cols) {
        Elem<float>::load8(p + c0, v);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        v[j] = c0 + j < cols ? p[c0 + j] : 0.0f;
}

// Eight values of z = BF16(x + residual) (x itself without a residual).
__device__ __forceinline__ uint4 add_bf16(const uint4 &a, const uint4 &b)
{
    return make_uint4(to_bf16x2(bf16_lo(a.x) + bf16_lo(b.x), bf16_hi(a.x) + bf16_hi(b.x)),
                      to_bf16x2(bf16_lo(a.y) + bf16_lo(b.y), bf16_hi(a.y) + bf16_hi(b.y)),
                      to_bf16x2(bf16_lo(a.z) + bf16_lo(b.z), bf16_hi(a.z) + bf16_hi(b.z)),
                      to_bf16x2(bf16_lo(a.w) + bf16_lo(b.w), bf16_hi(a.w) + bf16_hi(b.w)));
}

// Where a tile's (or a row's) codes and scales go.
struct QuantOut {
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t lds;   // scale row stride
};

// ---------------------------------------------------------------------------
// Quantise a 128-token x 128-column tile both ways from FP32 values.  Thread t
// owns columns 8 (t % 16) .. +7 of the 4 tokens 4 (t / 16) .. +3; a tile's
// values outside the tensor are zero.  Row amax: 16-lane DPP max.  Column
// amax: over the thread's tokens, the wave's four token groups, then the
// eight waves through LDS.  Four tokens' codes of a column are one 32-bit
// word of the LDS tile, written out as 128-byte rows.
// ---------------------------------------------------------------------------
struct TileShared {
    float red[TT / 64][128];
    float scl[128], rcl[128];
    uint32_t tile[128][32 + 1];   // [column][token / 4], odd stride
};

template <bool SLOW>
__device__ __forceinline__ void tile_codes(const float (&v)[4][8], const float (&srow)[4], const QuantOut &ro,
                                           int transpose_out, const QuantOut &to, int64_t tok0, int64_t col0,
                                           int64_t tokens, int64_t cols, bool full, TileShared &sh)
{
    const int t = threadIdx.x, cc = t & 15, rq = t >> 4;
    const int64_t c0 = col0 + 8 * cc;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t tk = tok0 + 4 * rq + i;
        const float s = srow[i], r = scale_inv(s);
        const uint32_t lo = codes4<SLOW>(v[i][0], v[i][1], v[i][2], v[i][3], s, r);
        const uint32_t hi = codes4<SLOW>(v[i][4], v[i][5], v[i][6], v[i][7], s, r);
        if (full)
            store_nt(ro.q + tk * ro.ldq + c0, lo, hi);
        else if (tk < tokens)
            store8_codes(ro.q + tk * ro.ldq, c0, cols, lo, hi);
    }
    uint32_t word[8];
#pragma unroll
    for (int j = 0; j < 8; j++)
        word[j] = codes4<SLOW>(v[0][j], v[1][j], v[2][j], v[3][j], sh.scl[8 * cc + j], sh.rcl[8 * cc + j]);
    if (!transpose_out) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t tk = tok0 + 4 * rq + i;
            uint32_t b[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                b[j] = (word[j] >> (8 * i)) & 0xFFu;
            const uint32_t lo = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
            const uint32_t hi = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
            if (tk < tokens)
                store8_codes(to.q + tk * to.ldq, c0, cols, lo, hi);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        sh.tile[8 * cc + j][rq] = word[j];
}

__device__ __forceinline__ void quant_tile(const float (&v)[4][8], const QuantOut &ro, int transpose_out,
                                           const QuantOut &to, int64_t tok0, int64_t col0, int64_t tokens,
                                           int64_t cols, int pow2, bool full, TileShared &sh)
{
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int cc = t & 15, rq = t >> 4;
    const int64_t bx = col0 >> 7, by = tok0 >> 7;
    bool slow = false;

    float m[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        float a = fmaxf(fmaxf(fabsf(v[0][j]), fabsf(v[1][j])), fmaxf(fabsf(v[2][j]), fabsf(v[3][j])));
        a = fmaxf(a, __shfl_xor(a, 16, 64));
        m[j] = fmaxf(a, __shfl_xor(a, 32, 64));
    }
    if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            sh.red[wave][8 * lane + j] = m[j];
    }
    float srow[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float a = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j++)
            a = fmaxf(a, fabsf(v[i][j]));
        srow[i] = block_scale(max16(a), pow2);
        slow = slow || scale_slow(srow[i]);
        const int64_t tk = tok0 + 4 * rq + i;
        if (cc == 0 && tk < tokens)
            ro.s[tk * ro.lds + bx] = srow[i];
    }
    __syncthreads();
    if (t < 128) {
        float a = sh.red[0][t];
#pragma unroll
        for (int k = 1; k < TT / 64; k++)
            a = fmaxf(a, sh.red[k][t]);
        const float s = block_scale(a, pow2);
        sh.scl[t] = s;
        sh.rcl[t] = scale_inv(s);
        slow = slow || scale_slow(s);
        const int64_t c = col0 + t;
        if (c < cols) {
            if (transpose_out)
                to.s[c * to.lds + by] = s;
            else
                to.s[by * to.lds + c] = s;
        }
    }
    if (__syncthreads_or(slow))
        tile_codes<true>(v, srow, ro, transpose_out, to, tok0, col0, tokens, cols, full, sh);
    else
        tile_codes<false>(v, srow, ro, transpose_out, to, tok0, col0, tokens, cols, full, sh);
    if (!transpose_out)
        return;
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 2; it++) {
        const int chunk = t + TT * it;
        const int row = chunk >> 3, seg = chunk & 7;
        const int64_t c = col0 + row, tk = tok0 + seg * 16;
        const uint32_t *src = &sh.tile[row][seg * 4];
        if (c >= cols)
            continue;
        uint8_t *dst = to.q + c * to.ldq + tk;
        if (tk + 16 <= tokens) {
            store_nt(dst, src[0], src[1], src[2], src[3]);
        } else {
            for (int e = 0; e < 16; e++)
                if (tk + e < tokens)
                    dst[e] = (uint8_t)(src[e >> 2] >> (8 * (e & 3)));
        }
    }
}

// Four rows x eight columns of a BF16 tensor for this thread (zeros outside).
__device__ __forceinline__ void load_tile(const uint16_t *x, int64_t ldx, int64_t tok0, int64_t col0, int64_t tokens,
                                          int64_t cols, bool full, uint4 (&a)[4])
{
    const int cc = threadIdx.x & 15, rq = threadIdx.x >> 4;
    const int64_t c0 = col0 + 8 * cc;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t tk = tok0 + 4 * rq + i;
        if (full)
            a[i] = *reinterpret_cast<const uint4 *>(x + tk * ldx + c0);
        else
            a[i] = tk < tokens ? load8_bf16(x + tk * ldx, c0, cols) : make_uint4(0, 0, 0, 0);
    }
}

// ---------------------------------------------------------------------------
// Row pass of the norm: one workgroup of NT threads per row.  Thread t holds
// columns 8 (t + NT k) .. +7, k < RUN, in registers; rows wider than
// 8 NT RUN read the rest of z a second time.  With QUANT the row's codes and
// scales are written too (the serving form); a 128-column block is 16
// consecutive lanes, so its amax is a DPP max.
// ---------------------------------------------------------------------------
constexpr int NT = 256, RUN = 4;

__device__ __forceinline__ float block_sum(float v, float *red)
{
    v = sum64(v);
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int i = 1; i < NT / 64; i++)
        s += red[i];
    return s;
}

template <bool QUANT>
__global__ __launch_bounds__(NT) void norm_row_kernel(const uint16_t *__restrict__ x, int64_t ldx,
                                                      const uint16_t *__restrict__ res, int64_t ldres,
                                                      const void *__restrict__ w, int wbf16, float eps, int64_t cols,
                                                      uint16_t *__restrict__ z, int64_t ldz,
                                                      float *__restrict__ rstd, uint16_t *__restrict__ h,
                                                      int64_t ldh, uint8_t *__restrict__ q, int64_t ldq,
                                                      float *__restrict__ s, int64_t nb, int pow2)
{
    __shared__ float red[NT / 64];
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x;
    const uint16_t *xr = x + row * ldx;
    const uint16_t *rr = res ? res + row * ldres : nullptr;
    uint16_t *zr = res ? z + row * ldz : nullptr;

    auto fetch = [&](int64_t c0) {
        uint4 a = load8_bf16(xr, c0, cols);
        if (rr) {
            a = add_bf16(a, load8_bf16(rr, c0, cols));
            const uint32_t o[4] = {a.x, a.y, a.z, a.w};
            store8_bf16(zr, c0, cols, o);
        }
        return a;
    };
    auto squares = [&](const uint4 &a) {
        float v[8], p = 0.0f;
        unpack8(a, v);
#pragma unroll
        for (int j = 0; j < 8; j++)
            p = fmaf(v[j], v[j], p);
        return p;
    };

    uint4 keep[RUN];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < RUN; k++) {
        const int64_t c0 = 8 * (int64_t)(t + NT * k);
        keep[k] = c0 < cols ? fetch(c0) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < RUN; k++)
        sum += squares(keep[k]);
    for (int64_t c0 = 8 * (int64_t)(t + NT * RUN); c0 < cols; c0 += 8 * NT)
        sum += squares(fetch(c0));
    const float r = 1.0f / sqrtf(block_sum(sum, red) / (float)cols + eps);
    if (t == 0 && rstd)
        rstd[row] = r;
    if constexpr (QUANT) {
        auto emit = [&](int64_t c0, const uint4 &a) {
            float n[8], wv[8], amax = 0.0f;
            unpack8(a, n);
            load8_weight(w, wbf16, c0, cols, wv);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                n[j] = n[j] * r * wv[j];
                amax = fmaxf(amax, fabsf(n[j]));
            }
            const float sc = block_scale(max16(amax), pow2), ri = scale_inv(sc);
            if (c0 >= cols)
                return;
            store8_codes(q + row * ldq, c0, cols, codes4<true>(n[0], n[1], n[2], n[3], sc, ri),
                         codes4<true>(n[4], n[5], n[6], n[7], sc, ri));
            if ((t & 15) == 0)
                s[row * nb + (c0 >> 7)] = sc;
            if (h) {
                const uint32_t o[4] = {to_bf16x2(n[0], n[1]), to_bf16x2(n[2], n[3]), to_bf16x2(n[4], n[5]),
                                       to_bf16x2(n[6], n[7])};
                store8_bf16(h + row * ldh, c0, cols, o);
            }
        };
        // every lane of a 16-lane group takes part in its block's max, past cols with zeros
        const int64_t span = (cols + 127) / 128 * 128;
#pragma unroll
        for (int k = 0; k < RUN; k++) {
            const int64_t c0 = 8 * (int64_t)(t + NT * k);
            if (c0 < span)
                emit(c0, keep[k]);
        }
        for (int64_t c0 = 8 * (int64_t)(t + NT * RUN); c0 < span; c0 += 8 * NT)
            emit(c0, rr ? (c0 < cols ? load8_bf16(zr, c0, cols) : make_uint4(0, 0, 0, 0))
                        : load8_bf16(xr, c0, cols));
    }
}

// Tile pass: n = z r w of a tile, quantised both ways (and stored as BF16
// when h is not NULL).
__global__ __launch_bounds__(TT) void norm_tile_kernel(const uint16_t *__restrict__ z, int64_t ldz,
                                                       const float *__restrict__ rstd, const void *__restrict__ w,
                                                       int wbf16, int64_t tokens, int64_t cols,
                                                       uint16_t *__restrict__ h, int64_t ldh, QuantOut ro,
                                                       int transpose_out, QuantOut to, int pow2)
{
    __shared__ TileShared sh;
    const int64_t tok0 = (int64_t)blockIdx.y * 128, col0 = (int64_t)blockIdx.x * 128;
    const bool full = tok0 + 128 <= tokens && col0 + 128 <= cols;
    const int cc = threadIdx.x & 15, rq = threadIdx.x >> 4;
    uint4 a[4];
    load_tile(z, ldz, tok0, col0, tokens, cols, full, a);
    float wv[8], v[4][8];
    load8_weight(w, wbf16, col0 + 8 * cc, cols, wv);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t tk = tok0 + 4 * rq + i;
        const float r = tk < tokens ? rstd[tk] : 0.0f;
        unpack8(a[i], v[i]);
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[i][j] = v[i][j] * r * wv[j];
        if (h && tk < tokens) {
            const uint32_t o[4] = {to_bf16x2(v[i][0], v[i][1]), to_bf16x2(v[i][2], v[i][3]),
                                   to_bf16x2(v[i][4], v[i][5]), to_bf16x2(v[i][6], v[i][7])};
            store8_bf16(h + tk * ldh, col0 + 8 * cc, cols, o);
        }
    }
    quant_tile(v, ro, transpose_out, to, tok0, col0, tokens, cols, pow2, full, sh);
}

// ---------------------------------------------------------------------------
// Norm gradient, row pass: c_t = mean over the row of w dy z r.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(NT) void norm_bwd_row_kernel(const uint16_t *__restrict__ dy, int64_t lddy,
                                                          const uint16_t *__restrict__ z, int64_t ldz,
                                                          const float *__restrict__ rstd,
                                                          const void *__restrict__ w, int wbf16, int64_t cols,
                                                          float *__restrict__ coef)
{
    __shared__ float red[NT / 64];
    const int64_t row = blockIdx.x;
    const uint16_t *dr = dy + row * lddy, *zr = z + row * ldz;
    float sum = 0.0f;
    for (int64_t c0 = 8 * (int64_t)threadIdx.x; c0 < cols; c0 += 8 * NT) {
        float d[8], v[8], wv[8];
        unpack8(load8_bf16(dr, c0, cols), d);
        unpack8(load8_bf16(zr, c0, cols), v);
        load8_weight(w, wbf16, c0, cols, wv);
#pragma unroll
        for (int j = 0; j < 8; j++)
            sum = fmaf(d[j] * wv[j], v[j], sum);
    }
    const float total = block_sum(sum, red);
    if (threadIdx.x == 0)
        coef[row] = total * rstd[row] / (float)cols;
}

// Tile pass: dx of a tile, stored as BF16 and quantised both ways, and the
// tile's share of dw (its 128 tokens), to part[token tile][column].
__global__ __launch_bounds__(TT) void norm_bwd_tile_kernel(const uint16_t *__restrict__ dy, int64_t lddy,
                                                           const uint16_t *__restrict__ z, int64_t ldz,
                                                           const float *__restrict__ rstd,
                                                           const float *__restrict__ coef,
                                                           const void *__restrict__ w, int wbf16,
                                                           const uint16_t *__restrict__ dres, int64_t lddres,
                                                           int64_t tokens, int64_t cols,
                                                           uint16_t *__restrict__ dx, int64_t lddx, QuantOut ro,
                                                           int transpose_out, QuantOut to,
                                                           float *__restrict__ part, int pow2)
{
    __shared__ TileShared sh;
    const int64_t tok0 = (int64_t)blockIdx.y * 128, col0 = (int64_t)blockIdx.x * 128;
    const bool full = tok0 + 128 <= tokens && col0 + 128 <= cols;
    const int t = threadIdx.x, cc = t & 15, rq = t >> 4, lane = t & 63, wave = t >> 6;
    uint4 a[4], b[4], d[4];
    load_tile(dy, lddy, tok0, col0, tokens, cols, full, a);
    load_tile(z, ldz, tok0, col0, tokens, cols, full, b);
    if (dres)
        load_tile(dres, lddres, tok0, col0, tokens, cols, full, d);
    float wv[8], v[4][8], dw[8];
    load8_weight(w, wbf16, col0 + 8 * cc, cols, wv);
#pragma unroll
    for (int j = 0; j < 8; j++)
        dw[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int64_t tk = tok0 + 4 * rq + i;
        const float r = tk < tokens ? rstd[tk] : 0.0f, ct = tk < tokens ? coef[tk] : 0.0f;
        float y[8], x[8], e[8];
        unpack8(a[i], y);
        unpack8(b[i], x);
        if (dres)
            unpack8(d[i], e);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float xh = x[j] * r;
            dw[j] = fmaf(y[j], xh, dw[j]);
            const float g = r * fmaf(-xh, ct, y[j] * wv[j]);
            v[i][j] = dres ? g + e[j] : g;
        }
        if (tk < tokens) {
            const uint32_t o[4] = {to_bf16x2(v[i][0], v[i][1]), to_bf16x2(v[i][2], v[i][3]),
                                   to_bf16x2(v[i][4], v[i][5]), to_bf16x2(v[i][6], v[i][7])};
            store8_bf16(dx + tk * lddx, col0 + 8 * cc, cols, o);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        dw[j] += __shfl_xor(dw[j], 16, 64);
        dw[j] += __shfl_xor(dw[j], 32, 64);
    }
    if (lane < 16) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            sh.red[wave][8 * lane + j] = dw[j];
    }
    __syncthreads();
    if (t < 128 && col0 + t < cols) {
        float s = sh.red[0][t];
#pragma unroll
        for (int k = 1; k < TT / 64; k++)
            s += sh.red[k][t];
        part[(int64_t)blockIdx.y * cols + col0 + t] = s;
    }
    __syncthreads();   // red is reused by the tile's column maxima
    quant_tile(v, ro, transpose_out, to, tok0, col0, tokens, cols, pow2, full, sh);
}

// dw = (dw +) the token tiles' shares, added in order.
__global__ __launch_bounds__(64) void norm_dw_kernel(const float *__restrict__ part, int64_t ntb, int64_t cols,
                                                     float *__restrict__ dw, int accumulate)
{
    const int64_t c = (int64_t)blockIdx.x * 64 + threadIdx.x;
    if (c >= cols)
        return;
    float s = 0.0f;
    for (int64_t k = 0; k < ntb; k++)
        s += part[k * cols + c];
    dw[c] = accumulate ? dw[c] + s : s;
}

// ---------------------------------------------------------------------------
// Gradient of h = silu(g) u.  With e = exp(-|g|) in (0, 1], sigmoid(g) and
// 1 - sigmoid(g) are 1 / (1 + e) and e / (1 + e), which one by the sign of g:
// neither overflows nor cancels.
//   du = dh g sigmoid(g),  dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g)))
// ---------------------------------------------------------------------------
__device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float &dg, float &du)
{
    const float e = expf(-fabsf(g));
    const float i = __builtin_amdgcn_rcpf(1.0f + e), ei = e * i;
    const float sig = g < 0.0f ? ei : i, nsig = g < 0.0f ? i : ei;
    du = dh * (g * sig);
    dg = (dh * u) * (sig * fmaf(g, nsig, 1.0f));
}

__global__ __launch_bounds__(TT) void swiglu_bwd_kernel(const uint16_t *__restrict__ dh, int64_t lddh,
                                                        const uint16_t *__restrict__ g, int64_t ldg,
                                                        const uint16_t *__restrict__ u, int64_t ldu, int64_t tokens,
                                                        int64_t cols, QuantOut gr, QuantOut ur, int transpose_out,
                                                        QuantOut gt, QuantOut ut, int pow2)
{
    __shared__ TileShared sh;
    const int64_t tok0 = (int64_t)blockIdx.y * 128, col0 = (int64_t)blockIdx.x * 128;
    const bool full = tok0 + 128 <= tokens && col0 + 128 <= cols;
    uint4 a[4], b[4], c[4];
    load_tile(dh, lddh, tok0, col0, tokens, cols, full, a);
    load_tile(g, ldg, tok0, col0, tokens, cols, full, b);
    load_tile(u, ldu, tok0, col0, tokens, cols, full, c);
    float vg[4][8], vu[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float x[8], y[8], w[8];
        unpack8(a[i], x);
        unpack8(b[i], y);
        unpack8(c[i], w);
#pragma unroll
        for (int j = 0; j < 8; j++)
            swiglu_grad(x[j], y[j], w[j], vg[i][j], vu[i][j]);
    }
    quant_tile(vg, gr, transpose_out, gt, tok0, col0, tokens, cols, pow2, full, sh);
    __syncthreads();   // the LDS tile of one gradient is read out before the other's is built
    quant_tile(vu, ur, transpose_out, ut, tok0, col0, tokens, cols, pow2, full, sh);
}

dim3 tile_grid(int64_t tokens, int64_t cols)
{
    return dim3((unsigned)((cols + 127) / 128), (unsigned)((tokens + 127) / 128));
}

} // namespace

hipError_t launch_norm_act(const NormIn &in, uint8_t *q, int64_t ldq, float *s, bool pow2, hipStream_t st)
{
    hipLaunchKernelGGL((norm_row_kernel<true>), dim3((unsigned)in.tokens), dim3(NT), 0, st, in.x, in.ldx, in.res,
                       in.ldres, in.w, (int)in.wbf16, in.eps, in.cols, in.z, in.ldz, in.rstd, in.h, in.ldh, q, ldq, s,
                       (in.cols + 127) / 128, (int)pow2);
    return hipGetLastError();
}

hipError_t launch_norm_dual(const NormIn &in, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                            int64_t ldqt, float *stok, bool pow2, hipStream_t st)
{
    const int64_t nb = (in.cols + 127) / 128, ntb = (in.tokens + 127) / 128;
    hipLaunchKernelGGL((norm_row_kernel<false>), dim3((unsigned)in.tokens), dim3(NT), 0, st, in.x, in.ldx, in.res,
                       in.ldres, in.w, (int)in.wbf16, in.eps, in.cols, in.z, in.ldz, in.rstd, nullptr, 0, nullptr, 0,
                       nullptr, nb, (int)pow2);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    hipLaunchKernelGGL(norm_tile_kernel, tile_grid(in.tokens, in.cols), dim3(TT), 0, st, in.res ? in.z : in.x,
                       in.res ? in.ldz : in.ldx, in.rstd, in.w, (int)in.wbf16, in.tokens, in.cols, in.h, in.ldh,
                       QuantOut{qr, ldqr, sr, nb}, (int)transpose_out,
                       QuantOut{qt, ldqt, stok, transpose_out ? ntb : in.cols}, (int)pow2);
    return hipGetLastError();
}

static size_t coef_bytes(int64_t tokens) { return ((size_t)tokens * 4 + 255) / 256 * 256; }

size_t norm_bwd_workspace_bytes(int64_t tokens, int64_t cols)
{
    return coef_bytes(tokens) + (size_t)((tokens + 127) / 128) * (size_t)cols * 4;
}

hipError_t launch_norm_bwd(const NormBwd &b, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                           int64_t ldqt, float *stok, bool pow2, void *workspace, hipStream_t st)
{
    const int64_t nb = (b.cols + 127) / 128, ntb = (b.tokens + 127) / 128;
    float *coef = (float *)workspace;
    float *part = (float *)((char *)workspace + coef_bytes(b.tokens));
    if (b.tokens > 0) {
        hipLaunchKernelGGL(norm_bwd_row_kernel, dim3((unsigned)b.tokens), dim3(NT), 0, st, b.dy, b.lddy, b.z, b.ldz,
                           b.rstd, b.w, (int)b.wbf16, b.cols, coef);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        hipLaunchKernelGGL(norm_bwd_tile_kernel, tile_grid(b.tokens, b.cols), dim3(TT), 0, st, b.dy, b.lddy, b.z,
                           b.ldz, b.rstd, coef, b.w, (int)b.wbf16, b.dres, b.lddres, b.tokens, b.cols, b.dx, b.lddx,
                           QuantOut{qr, ldqr, sr, nb}, (int)transpose_out,
                           QuantOut{qt, ldqt, stok, transpose_out ? ntb : b.cols}, part, (int)pow2);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((b.cols + 63) / 64)), dim3(64), 0, st, part, ntb, b.cols,
                       b.dw, (int)b.accumulate);
    return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwd &b, bool transpose_out, bool pow2, hipStream_t st)
{
    auto out = [](const GradOut &o, bool tok) {
        return tok ? QuantOut{o.q_tok, o.ldq_tok, o.s_tok, o.lds_tok} : QuantOut{o.q_row, o.ldq_row, o.s_row, o.lds_row};
    };
    hipLaunchKernelGGL(swiglu_bwd_kernel, tile_grid(b.tokens, b.cols), dim3(TT), 0, st, b.dh, b.lddh, b.g, b.ldg, b.u,
                       b.ldu, b.tokens, b.cols, out(b.dgate, false), out(b.dup, false), (int)transpose_out,
                       out(b.dgate, true), out(b.dup, true), (int)pow2);
    return hipGetLastError();
}

} // namespace puro
