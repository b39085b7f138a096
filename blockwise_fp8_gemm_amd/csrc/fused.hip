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
// All of them are HBM-bound (a copy moves 5.1 TB/s).  The token blocks of one
// column span 128 tokens and the norm's statistics a whole row, so the norm and
// its gradient take two passes: whole rows, then 128 x 128 tiles that hold one
// block of each kind per token and per column.  What the second pass reads again
// comes partly from the caches.  Small calls are launches: 2.6 us for a row of 2048.
#include "common.h"
#include "kernels.h"
#include "stores.h"

namespace puro {

namespace {

// A tile kernel's threads hold RT tokens x 8 columns each.  With two tokens and
// 1024 threads large tensors took longer (8192 x 2048 norm 12.1 against 9.2 us,
// its gradient 36.5 and 33.6; activation gradient of 8192 x 6144 147 and 112) and
// small ones little less (gradient of 700 x 1100: 9.2 against 10.7).
constexpr int RT = 4, TILE_THREADS = 16 * 128 / RT;

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

// max(|a|, |b|, m) for m >= 0, in one instruction (fmaxf would first quieten
// values that come straight from memory).
__device__ __forceinline__ float absmax3(float a, float b, float m)
{
    float r;
    asm("v_max3_f32 %0, |%1|, |%2|, %3" : "=v"(r) : "v"(a), "v"(b), "v"(m));
    return r;
}

// A block's scale s and its reciprocal r + rl, rl >= 0 the part that FP32 r
// lacks: v / s is then fma(v, r, v rl), two operations, within 0.5 + 2^-20 ulps of
// the quotient (rl >= 0 keeps the sign of -0).  s = amax / 448 by one
// correction step from 1/448's FP32 value, exact as IEEE division while the
// residual does not underflow.  r = 0 for a zero scale (codes +-0 by sign).  A
// scale below 2^-96, whose reciprocal could overflow, has that of s 2^64 and
// its values are multiplied by 2^64 first (exact: they are at most 671 s, see
// below), which SLOW selects for a whole tile or run.  There a subnormal scale of
// few bits can lie a third below amax / 448 (amax = 671 x 2^-149 has the scale
// 2^-149), so the quotient is limited to +-448 before the cast.
struct Scale {
    float s, r, rl;
};
__device__ __forceinline__ bool scale_tiny(float s) { return s < 0x1p-96f; }
__device__ __forceinline__ bool scale_slow(float s, int pow2) { return !pow2 && s != 0.0f && scale_tiny(s); }

__device__ __forceinline__ Scale make_scale(float amax, int pow2)
{
    Scale o;
    if (pow2) {
        o.s = pow2_scale(amax);
        o.r = __uint_as_float(0x7F000000u - (__float_as_uint(o.s) & 0x7F800000u));
        o.rl = 0.0f;
        return o;
    }
    const float c = 1.0f / 448.0f, q = amax * c;
    o.s = fmaf(fmaf(-q, 448.0f, amax), c, q);
    if (amax < 0x1p-80f)
        o.s = amax / 448.0f;
    const float s = scale_tiny(o.s) ? o.s * 0x1p64f : o.s, r0 = __builtin_amdgcn_rcpf(s);
    float r = fmaf(fmaf(-s, r0, 1.0f), r0, r0), e = fmaf(-s, r, 1.0f);
    if (e < 0.0f) {   // r above 1 / s: the float below it
        r = __uint_as_float(__float_as_uint(r) - 1);
        e = fmaf(-s, r, 1.0f);
    }
    o.r = s > 0.0f ? r : 0.0f;
    o.rl = s > 0.0f ? e * r : 0.0f;
    return o;
}

template <bool SLOW> __device__ __forceinline__ float code_arg(float v, const Scale &c)
{
    if (SLOW)
        v = scale_tiny(c.s) ? v * 0x1p64f : v;
    const float y = fmaf(v, c.r, v * c.rl);
    return SLOW ? saturate(y) : y;
}

template <bool SLOW> __device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const Scale &s)
{
    return e4m3x4(code_arg<SLOW>(a, s), code_arg<SLOW>(b, s), code_arg<SLOW>(c, s), code_arg<SLOW>(d, s));
}

// The first n of 16 bytes (0 < n < 16) to a 16-byte aligned address, in at most
// four stores.
__device__ __forceinline__ void store_some(uint8_t *p, const uint32_t w[4], int n)
{
    uint32_t a = w[0], b = w[1];
    if (n & 8) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(a, b);
        a = w[2];
        b = w[3];
        p += 8;
    }
    if (n & 4) {
        *reinterpret_cast<uint32_t *>(p) = a;
        a = b;
        p += 4;
    }
    if (n & 2) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)a;
        a >>= 16;
        p += 2;
    }
    if (n & 1)
        *p = (uint8_t)a;
}

// Eight BF16 values of a row from column c0 on (a multiple of 8), zeros at and past cols.
__device__ __forceinline__ uint4 load8_bf16(const uint16_t *row, int64_t c0, int64_t cols)
{
    if (c0 + 8 <= cols)
        return *reinterpret_cast<const uint4 *>(row + c0);
    uint4 r = make_uint4(0, 0, 0, 0);
    if (c0 >= cols)
        return r;
    const int n = (int)(cols - c0);
    const uint16_t *p = row + c0;
    uint32_t two = 0, one = 0;
    if (n & 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.x = v.x;
        r.y = v.y;
    }
    if (n & 2)
        two = *reinterpret_cast<const uint32_t *>(p + (n & 4));
    if (n & 1)
        one = p[n & 6];
    const uint32_t lo = n & 2 ? two : one, hi = n & 2 ? one : 0;
    if (n & 4) {
        r.z = lo;
        r.w = hi;
    } else {
        r.x = lo;
        r.y = hi;
    }
    return r;
}

__device__ __forceinline__ void store8_bf16(uint16_t *row, int64_t c0, int64_t cols, const uint32_t w[4])
{
    if (c0 + 8 <= cols)
        store_nt(row + c0, w[0], w[1], w[2], w[3]);
    else if (c0 < cols)
        store_some(reinterpret_cast<uint8_t *>(row + c0), w, 2 * (int)(cols - c0));
}

__device__ __forceinline__ void store8_codes(uint8_t *row, int64_t c0, int64_t cols, uint32_t lo, uint32_t hi)
{
    if (c0 + 8 <= cols) {
        store_nt(row + c0, lo, hi);
    } else if (c0 < cols) {
        const uint32_t w[4] = {lo, hi, 0, 0};
        store_some(row + c0, w, (int)(cols - c0));
    }
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
// owns columns 8 (t % 16) .. +7 of the RT tokens RT (t / 16) .. + RT - 1; a
// tile's values outside the tensor are zero.  Row amax: 16-lane DPP max; lanes
// 0 .. RT - 1 of a 16-lane group then each form one token's scale.  Column amax:
// over the thread's tokens, the wave's four token groups (each exchange step
// halves the columns a lane carries on), then the waves through LDS.  The
// column codes are turned in LDS and written out as 128-byte rows.
// ---------------------------------------------------------------------------
struct TileShared {
    static constexpr int WAVES = TILE_THREADS / 64;
    float red[WAVES][128];
    float scl[128], rcl[128], rll[128];   // column scales, reciprocals and their low parts
    uint32_t slow[WAVES];                 // whether a wave met a scale below 2^-96
    uint8_t tile[128][128 + 4];           // [column][token] codes, odd stride in dwords
};

// Holds the compiler to forming a tile's values here, once: left alone it
// carries the factors of each value along and forms it again at every use,
// which takes more registers than the values themselves and spills.
__device__ __forceinline__ void pin(float (&v)[RT][8])
{
#pragma unroll
    for (int i = 0; i < RT; i++)
#pragma unroll
        for (int j = 0; j < 8; j++)
            asm volatile("" : "+v"(v[i][j]));
}

// This thread's place in a tile.
struct Place {
    int64_t tok0, col0, tokens, cols;
    int cc, rq;
    __device__ __forceinline__ int64_t tk(int i) const { return tok0 + RT * rq + i; }
    __device__ __forceinline__ int64_t c0() const { return col0 + 8 * cc; }
};
// Tiles are taken row by row (measured against eight neighbours per XCD, which
// saves partial sectors of the row scales: 5 to 8% slower).
__device__ __forceinline__ Place place(unsigned row, unsigned col, int64_t tokens, int64_t cols)
{
    return Place{(int64_t)row * 128, (int64_t)col * 128, tokens, cols, (int)threadIdx.x & 15,
                     (int)threadIdx.x >> 4};
}

// Exchange between the wave's halves, then between its 16-lane rows: op over
// the four lanes with equal lane % 16 of eight values; lane group g = lane / 16
// ends with the results of values first(g) and first(g) + 1.
__device__ __forceinline__ int first_of(int lane) { return ((lane >> 5) & 1) * 4 + ((lane >> 4) & 1) * 2; }
template <class Op> __device__ __forceinline__ float2 cross4(const float (&m)[8], Op op)
{
    float p[4], q[2];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(m[k]), __float_as_uint(m[k + 4]), false, false);
        p[k] = op(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
        const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(p[k]), __float_as_uint(p[k + 2]), false, false);
        q[k] = op(__uint_as_float(x[0]), __uint_as_float(x[1]));
    }
    return make_float2(q[0], q[1]);
}

template <int I> __device__ __forceinline__ Scale row_scale(const Scale &own)
{
    return Scale{dpp_f<0x150 + I>(own.s), dpp_f<0x150 + I>(own.r), dpp_f<0x150 + I>(own.rl)};
}

template <bool SLOW, bool FULL, bool TR, bool ROWS>
__device__ __forceinline__ void tile_codes(const float (&v)[RT][8], const Scale &own, const QuantOut &ro,
                                           const QuantOut &to, const Place &p, TileShared &sh)
{
    if constexpr (ROWS) {
        const Scale sr[RT] = {row_scale<0>(own), row_scale<1>(own), row_scale<2>(own), row_scale<3>(own)};
        uint8_t *qr = ro.q + p.tk(0) * ro.ldq + (FULL ? p.c0() : 0);
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const uint32_t lo = codes4<SLOW>(v[i][0], v[i][1], v[i][2], v[i][3], sr[i]);
            const uint32_t hi = codes4<SLOW>(v[i][4], v[i][5], v[i][6], v[i][7], sr[i]);
            if (FULL)
                store_nt(qr + i * ro.ldq, lo, hi);
            else if (p.tk(i) < p.tokens)
                store8_codes(qr + i * ro.ldq, p.c0(), p.cols, lo, hi);
        }
    }
    uint32_t word[8];   // RT codes of a column, a byte each
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const Scale c{SLOW ? sh.scl[8 * p.cc + j] : 0.0f, sh.rcl[8 * p.cc + j], sh.rll[8 * p.cc + j]};
        word[j] = codes4<SLOW>(v[0][j], v[1][j], v[2][j], v[3][j], c);
        if (SLOW)
            __builtin_amdgcn_sched_barrier(0);   // a column at a time: the wide form's temporaries do not fit several
    }
    if constexpr (!TR) {
#pragma unroll
        for (int i = 0; i < RT; i++) {
            uint32_t b[8];
#pragma unroll
            for (int j = 0; j < 8; j++)
                b[j] = (word[j] >> (8 * i)) & 0xFFu;
            const uint32_t lo = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
            const uint32_t hi = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
            if (p.tk(i) < p.tokens)
                store8_codes(to.q + p.tk(i) * to.ldq, p.c0(), p.cols, lo, hi);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        *reinterpret_cast<uint32_t *>(&sh.tile[8 * p.cc + j][RT * p.rq]) = word[j];
}

template <bool FULL, bool TR, bool ROWS>
__device__ __forceinline__ void quant_tile(const float (&v)[RT][8], const QuantOut &ro, const QuantOut &to,
                                           const Place &p, int pow2, TileShared &sh)
{
    constexpr int WAVES = TileShared::WAVES;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t bx = p.col0 >> 7, by = p.tok0 >> 7;

    float m[8];
#pragma unroll
    for (int j = 0; j < 8; j++)
        m[j] = absmax3(v[2][j], v[3][j], absmax3(v[0][j], v[1][j], 0.0f));
    *reinterpret_cast<float2 *>(&sh.red[wave][8 * p.cc + first_of(lane)]) =
        cross4(m, [](float a, float b) { return absmax3(a, b, 0.0f); });
    Scale own{0.0f, 0.0f, 0.0f};
    uint32_t slow = 0;
    if constexpr (ROWS) {
        float a[RT];
#pragma unroll
        for (int i = 0; i < RT; i++)
            a[i] = max16(absmax3(v[i][6], v[i][7], absmax3(v[i][4], v[i][5], absmax3(v[i][2], v[i][3],
                         absmax3(v[i][0], v[i][1], 0.0f)))));
        own = make_scale(p.cc & 2 ? (p.cc & 1 ? a[3] : a[2]) : (p.cc & 1 ? a[1] : a[0]), pow2);
        slow = __any(scale_slow(own.s, pow2));
        if (p.cc < RT && (FULL || p.tk(p.cc) < p.tokens))
            ro.s[p.tk(p.cc) * ro.lds + bx] = own.s;
    }
    __syncthreads();
    if (t < 128) {
        float c = sh.red[0][t];
#pragma unroll
        for (int k = 1; k < WAVES; k++)
            c = absmax3(c, sh.red[k][t], 0.0f);
        const Scale o = make_scale(c, pow2);
        sh.scl[t] = o.s;
        sh.rcl[t] = o.r;
        sh.rll[t] = o.rl;
        slow |= __any(scale_slow(o.s, pow2));
        if (FULL || p.col0 + t < p.cols) {
            if (TR)
                to.s[(p.col0 + t) * to.lds + by] = o.s;
            else
                to.s[by * to.lds + p.col0 + t] = o.s;
        }
    }
    if (lane == 0)
        sh.slow[wave] = slow;
    __syncthreads();
    slow = 0;
#pragma unroll
    for (int k = 0; k < WAVES; k++)
        slow |= sh.slow[k];
    if (__builtin_amdgcn_readfirstlane(slow))
        tile_codes<true, FULL, TR, ROWS>(v, own, ro, to, p, sh);
    else
        tile_codes<false, FULL, TR, ROWS>(v, own, ro, to, p, sh);
    if (!TR)
        return;
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 1024 / TILE_THREADS; it++) {
        const int chunk = t + TILE_THREADS * it;
        const int row = chunk >> 3, seg = chunk & 7;
        const int64_t c = p.col0 + row, tk = p.tok0 + seg * 16;
        const uint32_t *src = reinterpret_cast<const uint32_t *>(&sh.tile[row][seg * 16]);
        uint8_t *dst = to.q + c * to.ldq + tk;
        if (FULL || (c < p.cols && tk + 16 <= p.tokens)) {
            store_nt(dst, src[0], src[1], src[2], src[3]);
        } else if (c < p.cols && tk < p.tokens) {
            const uint32_t w[4] = {src[0], src[1], src[2], src[3]};
            store_some(dst, w, (int)(p.tokens - tk));
        }
    }
}

// RT rows x eight columns of a BF16 tensor for this thread (zeros outside).
template <bool FULL>
__device__ __forceinline__ void load_tile(const uint16_t *x, int64_t ldx, const Place &p, uint4 (&a)[RT])
{
    const uint16_t *row = x + p.tk(0) * ldx;
#pragma unroll
    for (int i = 0; i < RT; i++) {
        if (FULL)
            a[i] = *reinterpret_cast<const uint4 *>(row + i * ldx + p.c0());
        else
            a[i] = p.tk(i) < p.tokens ? load8_bf16(row + i * ldx, p.c0(), p.cols) : make_uint4(0, 0, 0, 0);
    }
}

template <bool FULL>
__device__ __forceinline__ void store_tile(uint16_t *x, int64_t ldx, const Place &p, const float (&v)[RT][8])
{
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const uint32_t o[4] = {to_bf16x2(v[i][0], v[i][1]), to_bf16x2(v[i][2], v[i][3]), to_bf16x2(v[i][4], v[i][5]),
                               to_bf16x2(v[i][6], v[i][7])};
        if (FULL)
            store_nt(x + p.tk(i) * ldx + p.c0(), o[0], o[1], o[2], o[3]);
        else if (p.tk(i) < p.tokens)
            store8_bf16(x + p.tk(i) * ldx, p.c0(), p.cols, o);
    }
}

// Whole tiles (uniform over the workgroup) and edge tiles are two bodies of one kernel.
__device__ __forceinline__ bool full_tile(const Place &p)
{
    return p.tok0 + 128 <= p.tokens && p.col0 + 128 <= p.cols;
}

// ---------------------------------------------------------------------------
// Row pass of the norm: a workgroup of NT threads takes every gridDim-th row.
// Thread t holds columns 8 (t + NT k) .. +7, k < RUN, of the row and their
// weights in registers, and has the next row's loads in flight while it works
// on this one; rows wider than 8 NT RUN read the rest of z a second time.  The
// row's codes and scales are written here (all there is in the serving form): a
// 128-column block is 16 consecutive lanes, so its amax is a DPP max.  8192 x 2048
// with a residual: 20.7 us for 118 MB, 5.7 TB/s; 1037 x 2048: 5.5 us.
// ---------------------------------------------------------------------------
constexpr int NT = 256;

// Sum over the workgroup; `red` may be used again after the call after next.
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

__device__ __forceinline__ float squares(const uint4 &a)
{
    float v[8], p = 0.0f;
    unpack8(a, v);
#pragma unroll
    for (int j = 0; j < 8; j++)
        p = fmaf(v[j], v[j], p);
    return p;
}

template <int RUN>
__global__ __launch_bounds__(NT) void norm_row_kernel(NormIn in, uint8_t *__restrict__ q, int64_t ldq,
                                                      float *__restrict__ s, int64_t nb, int pow2, int keep_z)
{
    constexpr bool WIDE = RUN == 4;   // rows that do not fit the registers reach the widest form only
    __shared__ float red[2][NT / 64];
    const int t = threadIdx.x;
    const int64_t cols = in.cols, span = nb * 128;
    const bool res = in.res != nullptr;

    float w[RUN][8];
    uint4 x[RUN], r[RUN];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int k = 0; k < RUN; k++) {
            const int64_t c0 = 8 * (int64_t)(t + NT * k);
            x[k] = load8_bf16(in.x + row * in.ldx, c0, cols);
            if (res)
                r[k] = load8_bf16(in.res + row * in.ldres, c0, cols);
        }
    };
    auto emit = [&](int64_t row, int64_t c0, const uint4 &a, const float (&wv)[8], float rs) {
        float n[8];
        unpack8(a, n);
#pragma unroll
        for (int j = 0; j < 8; j++)
            n[j] = n[j] * rs * wv[j];
        const Scale sc = make_scale(max16(absmax3(n[6], n[7], absmax3(n[4], n[5], absmax3(n[2], n[3],
                                          absmax3(n[0], n[1], 0.0f))))), pow2);
        uint32_t lo, hi;
        if (__any(scale_slow(sc.s, pow2))) {
            lo = codes4<true>(n[0], n[1], n[2], n[3], sc);
            hi = codes4<true>(n[4], n[5], n[6], n[7], sc);
        } else {
            lo = codes4<false>(n[0], n[1], n[2], n[3], sc);
            hi = codes4<false>(n[4], n[5], n[6], n[7], sc);
        }
        store8_codes(q + row * ldq, c0, cols, lo, hi);
        if ((t & 15) == 0)
            s[row * nb + (c0 >> 7)] = sc.s;
        if (in.h) {
            const uint32_t o[4] = {to_bf16x2(n[0], n[1]), to_bf16x2(n[2], n[3]), to_bf16x2(n[4], n[5]),
                                   to_bf16x2(n[6], n[7])};
            store8_bf16(in.h + row * in.ldh, c0, cols, o);
        }
    };

    fetch(blockIdx.x);
#pragma unroll
    for (int k = 0; k < RUN; k++)
        load8_weight(in.w, in.wbf16, 8 * (int64_t)(t + NT * k), cols, w[k]);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < in.tokens; row += gridDim.x, turn ^= 1) {
        const uint16_t *xr = in.x + row * in.ldx, *rr = in.res + row * in.ldres;
        uint16_t *zr = in.z + row * in.ldz;
        auto sum_and_store = [&](uint4 &a, const uint4 &b, int64_t c0) {
            if (res) {
                a = add_bf16(a, b);
                const uint32_t o[4] = {a.x, a.y, a.z, a.w};
                if (keep_z && c0 + 8 <= cols)
                    *reinterpret_cast<uint4 *>(zr + c0) = a;
                else
                    store8_bf16(zr, c0, cols, o);
            }
            return squares(a);
        };
        uint4 z[RUN];
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < RUN; k++) {
            z[k] = x[k];
            sum += sum_and_store(z[k], r[k], 8 * (int64_t)(t + NT * k));
        }
        for (int64_t c0 = 8 * (int64_t)(t + NT * RUN); WIDE && c0 < cols; c0 += 8 * NT) {
            uint4 a = load8_bf16(xr, c0, cols);
            sum += sum_and_store(a, res ? load8_bf16(rr, c0, cols) : a, c0);
        }
        if (row + gridDim.x < in.tokens)
            fetch(row + gridDim.x);
        const float rs = 1.0f / sqrtf(block_sum(sum, red[turn]) / (float)cols + in.eps);
        if (t == 0 && in.rstd)
            in.rstd[row] = rs;
        // every lane of a 16-lane group takes part in its block's max, past cols with zeros
#pragma unroll
        for (int k = 0; k < RUN; k++) {
            const int64_t c0 = 8 * (int64_t)(t + NT * k);
            if (c0 < span)
                emit(row, c0, z[k], w[k], rs);
        }
        for (int64_t c0 = 8 * (int64_t)(t + NT * RUN); WIDE && c0 < span; c0 += 8 * NT) {
            float wv[8];
            load8_weight(in.w, in.wbf16, c0, cols, wv);
            emit(row, c0, load8_bf16(res ? zr : xr, c0, cols), wv, rs);
        }
    }
}

// Tile pass: n = z r w of a tile, formed again and quantised along the tokens
// (8192 x 2048: 9.2 us, 51 MB).  The row pass has a row in registers and writes
// its codes: with those written here too both passes took 36.9 us instead of 31.7.
template <bool FULL, bool TR>
__device__ __forceinline__ void norm_tile(const uint16_t *z, int64_t ldz, const float *rstd, const void *w, int wbf16,
                                          const Place &p, const QuantOut &to, int pow2, TileShared &sh)
{
    uint4 a[RT];
    load_tile<FULL>(z, ldz, p, a);
    float wv[8], v[RT][8];
    load8_weight(w, wbf16, p.c0(), p.cols, wv);
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const float r = FULL || p.tk(i) < p.tokens ? rstd[p.tk(i)] : 0.0f;
        unpack8(a[i], v[i]);
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[i][j] = v[i][j] * r * wv[j];
    }
    pin(v);
    quant_tile<FULL, TR, false>(v, QuantOut{}, to, p, pow2, sh);
}

template <bool TR>
__global__ __launch_bounds__(TILE_THREADS) __attribute__((amdgpu_waves_per_eu(5)))
void norm_tile_kernel(const uint16_t *__restrict__ z, int64_t ldz, const float *__restrict__ rstd,
                      const void *__restrict__ w, int wbf16, int64_t tokens, int64_t cols, QuantOut to, int pow2)
{
    __shared__ TileShared sh;
    const auto p = place(blockIdx.y, blockIdx.x, tokens, cols);
    if (full_tile(p))
        norm_tile<true, TR>(z, ldz, rstd, w, wbf16, p, to, pow2, sh);
    else
        norm_tile<false, TR>(z, ldz, rstd, w, wbf16, p, to, pow2, sh);
}

// ---------------------------------------------------------------------------
// Norm gradient.  Row pass, over every gridDim-th row like the norm's: c_t =
// mean over the row of w dy z r, and this workgroup's share of dw, its rows'
// dy z r, to part[workgroup][column] (rows of ldp, a multiple of 16).  8192 x
// 2048: 14.4 us for 76 MB.  Writing dx and its row codes here as well, with a tile
// pass for the token copy only, took 54 us for both passes against 48.
// ---------------------------------------------------------------------------
template <int RUN>
__global__ __launch_bounds__(NT) void norm_bwd_row_kernel(NormBwd b, float *__restrict__ coef,
                                                          float *__restrict__ part, int64_t ldp)
{
    constexpr bool WIDE = RUN == 4;   // rows that do not fit the registers reach the widest form only
    __shared__ float red[2][NT / 64];
    const int t = threadIdx.x;
    const int64_t cols = b.cols;
    float *mine = part + blockIdx.x * ldp;

    float w[RUN][8], dw[RUN][8];
    uint4 y[RUN], x[RUN];
    float rstd = 0.0f;
    auto fetch = [&](int64_t row) {
        rstd = b.rstd[row];
#pragma unroll
        for (int k = 0; k < RUN; k++) {
            const int64_t c0 = 8 * (int64_t)(t + NT * k);
            y[k] = load8_bf16(b.dy + row * b.lddy, c0, cols);
            x[k] = load8_bf16(b.z + row * b.ldz, c0, cols);
        }
    };
    // sum of w dy (z r), and dw += dy (z r): the factor r first, which brings z to order one, so that
    // neither leaves FP32's range where the result does not
    auto inner = [&](const uint4 &dy, const uint4 &z, const float (&wv)[8], float r, float (&acc)[8]) {
        float yv[8], xv[8], p = 0.0f;
        unpack8(dy, yv);
        unpack8(z, xv);
#pragma unroll
        for (int j = 0; j < 8; j++) {
            const float xh = xv[j] * r;
            p = fmaf(yv[j] * wv[j], xh, p);
            acc[j] = fmaf(yv[j], xh, acc[j]);
        }
        return p;
    };
    auto put = [&](int64_t c0, const float (&v)[8]) {
        *reinterpret_cast<float4 *>(mine + c0) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(mine + c0 + 4) = make_float4(v[4], v[5], v[6], v[7]);
    };

    fetch(blockIdx.x);
#pragma unroll
    for (int k = 0; k < RUN; k++) {
        load8_weight(b.w, b.wbf16, 8 * (int64_t)(t + NT * k), cols, w[k]);
#pragma unroll
        for (int j = 0; j < 8; j++)
            dw[k][j] = 0.0f;
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < b.tokens; row += gridDim.x, turn ^= 1) {
        const float r = rstd;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < RUN; k++)
            sum += inner(y[k], x[k], w[k], r, dw[k]);
        if (row + gridDim.x < b.tokens)
            fetch(row + gridDim.x);
        for (int64_t c0 = 8 * (int64_t)(t + NT * RUN); WIDE && c0 < cols; c0 += 8 * NT) {
            // columns past the registers: this workgroup's share of dw is kept in part itself
            float wv[8], acc[8];
            load8_weight(b.w, b.wbf16, c0, cols, wv);
            if (row == blockIdx.x) {
#pragma unroll
                for (int j = 0; j < 8; j++)
                    acc[j] = 0.0f;
            } else {
                Elem<float>::load8(mine + c0, acc);
            }
            sum += inner(load8_bf16(b.dy + row * b.lddy, c0, cols), load8_bf16(b.z + row * b.ldz, c0, cols), wv, r, acc);
            put(c0, acc);
        }
        const float total = block_sum(sum, red[turn]);
        if (t == 0)
            coef[row] = total / (float)cols;
    }
#pragma unroll
    for (int k = 0; k < RUN; k++) {
        const int64_t c0 = 8 * (int64_t)(t + NT * k);
        if (c0 < cols)
            put(c0, dw[k]);
    }
}

// Tile pass: dx of a tile, stored as BF16 and quantised both ways (8192 x 2048:
// 33.6 us for 182 MB, 5.4 TB/s).
template <bool FULL, bool TR>
__device__ __forceinline__ void norm_bwd_tile(const NormBwd &b, const float *coef, const Place &p,
                                              const QuantOut &ro, const QuantOut &to, int pow2, TileShared &sh)
{
    uint4 y[RT], z[RT], d[RT];
    load_tile<FULL>(b.dy, b.lddy, p, y);
    load_tile<FULL>(b.z, b.ldz, p, z);
    if (b.dres)
        load_tile<FULL>(b.dres, b.lddres, p, d);
    float wv[8], v[RT][8];
    load8_weight(b.w, b.wbf16, p.c0(), p.cols, wv);
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const bool in = FULL || p.tk(i) < p.tokens;
        const float r = in ? b.rstd[p.tk(i)] : 0.0f, ct = in ? coef[p.tk(i)] : 0.0f;
        float yv[8], x[8];
        unpack8(y[i], yv);
        unpack8(z[i], x);
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[i][j] = r * fmaf(-(x[j] * r), ct, yv[j] * wv[j]);
        if (b.dres) {
            float e[8];
            unpack8(d[i], e);
#pragma unroll
            for (int j = 0; j < 8; j++)
                v[i][j] += e[j];
        }
    }
    pin(v);
    store_tile<FULL>(b.dx, b.lddx, p, v);
    quant_tile<FULL, TR, true>(v, ro, to, p, pow2, sh);
}

// dw = (dw +) the workgroups' shares, for 32 columns: 16 threads per column take
// every 16th share, and their sums are added in a fixed order.
constexpr int DW_COLS = 32, DW_ROWS = TILE_THREADS / DW_COLS;
__device__ __forceinline__ void sum_dw(const float *part, int parts, int64_t ldp, int64_t cols, int64_t col0,
                                       float *dw, bool accumulate, float (*red)[DW_COLS])
{
    const int x = threadIdx.x % DW_COLS, y = threadIdx.x / DW_COLS;
    const int64_t c = col0 + x;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 8
        for (int k = y; k < parts; k += DW_ROWS)
            s += part[k * ldp + c];
    }
    red[y][x] = s;
    for (int n = DW_ROWS / 2; n > 0; n >>= 1) {
        __syncthreads();
        if (y < n)
            red[y][x] += red[y + n][x];
    }
    if (y == 0 && c < cols)
        dw[c] = accumulate ? dw[c] + red[0][x] : red[0][x];
}

// The first workgroups add up dw, the others take a tile each.  (One extent: the
// 2^16 rows of tiles that 2^23 tokens have are all that a grid's second one holds.)
__host__ __device__ inline unsigned dw_groups(int64_t cols) { return (unsigned)((cols + DW_COLS - 1) / DW_COLS); }
template <bool TR>
__global__ __launch_bounds__(TILE_THREADS) __attribute__((amdgpu_waves_per_eu(4)))
void norm_bwd_tile_kernel(NormBwd b, const float *__restrict__ coef, const float *__restrict__ part, int parts,
                          int64_t ldp, QuantOut ro, QuantOut to, int pow2)
{
    __shared__ TileShared sh;
    const unsigned sums = dw_groups(b.cols);
    if (blockIdx.x < sums) {
        sum_dw(part, parts, ldp, b.cols, (int64_t)blockIdx.x * DW_COLS, b.dw, b.accumulate,
               reinterpret_cast<float(*)[DW_COLS]>(&sh.red[0][0]));
        return;
    }
    const unsigned tile = blockIdx.x - sums, nb = (unsigned)((b.cols + 127) >> 7);
    const unsigned row = __builtin_amdgcn_readfirstlane(tile / nb);   // formed in a vector register
    const auto p = place(row, tile - row * nb, b.tokens, b.cols);
    if (full_tile(p))
        norm_bwd_tile<true, TR>(b, coef, p, ro, to, pow2, sh);
    else
        norm_bwd_tile<false, TR>(b, coef, p, ro, to, pow2, sh);
}

// ---------------------------------------------------------------------------
// Gradient of h = silu(g) u.  With e = exp(-|g|) in (0, 1], sigmoid(g) and
// 1 - sigmoid(g) are 1 / (1 + e) and e / (1 + e), which one by the sign of g:
// neither overflows nor cancels.
//   du = dh g sigmoid(g),  dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g)))
// e = 2^t, t = -|g| log2(e): what t rounds off (h + l, from the two-part
// constant) comes back as a factor 1 + l ln 2, and 1 / (1 + e) is v_rcp_f32's
// value with a correction step, so that the two cost one rounding each beside
// v_exp_f32's one step.  (e as the square of 2^(t / 2) and the bare reciprocal
// were 1.5 to 1.9 times as far from the exact values for negative gates, and
// 1% faster.)  v_exp_f32 gives 0 below its normal range: where one of a
// wave's gates is that far out (FAR), those take 2^(t + 64) 2^-64, which keeps e down
// to its subnormals; the others' values are the same bits in both forms.  One
// pass over tiles; 8192 x 6144: 110 us for 540 MB, of which 510 are the operands
// and results (row scales leave as partial sectors), 4.9 TB/s.  The 54 vector
// instructions an element takes with both its quantisations fill 0.6 of that time; a
// single tile alone on a CU takes 12 us.
// ---------------------------------------------------------------------------
constexpr float kNearGate = 87.0f;   // e^-87 = 2^-125.5
template <bool FAR> __device__ __forceinline__ void swiglu_grad(float dh, float g, float u, float &dg, float &du)
{
    // past 256 e is 0, and h must stay finite
    const float a = FAR ? fminf(fabsf(g), 256.0f) : fabsf(g), h = a * -0x1.715476p0f;
    const float l = fmaf(a, -0x1.4ae0cp-26f, fmaf(a, -0x1.715476p0f, -h));
    const bool far = FAR && h < -126.0f;
    const float x = __builtin_amdgcn_exp2f(far ? h + 64.0f : h), q = fmaf(x, l * 0x1.62e43p-1f, x);
    const float e = far ? q * 0x1p-64f : q;
    const float d = 1.0f + e, i0 = __builtin_amdgcn_rcpf(d), i = fmaf(fmaf(-d, i0, 1.0f), i0, i0), ei = e * i;
    const float sig = g < 0.0f ? ei : i, nsig = g < 0.0f ? i : ei;
    du = dh * (g * sig);
    dg = (dh * u) * (sig * fmaf(g, nsig, 1.0f));
}

template <bool FULL, bool TR>
__device__ __forceinline__ void swiglu_bwd_tile(const SwigluBwd &b, const Place &p, int pow2,
                                                TileShared &sh)
{
    uint4 x[RT], g[RT], u[RT];
    load_tile<FULL>(b.dh, b.lddh, p, x);
    load_tile<FULL>(b.g, b.ldg, p, g);
    load_tile<FULL>(b.u, b.ldu, p, u);
    float vg[RT][8], vu[RT][8];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        float xv[8], gv[8], uv[8];
        unpack8(x[i], xv);
        unpack8(g[i], gv);
        unpack8(u[i], uv);
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            m = absmax3(gv[j], gv[j + 1], m);
        if (__any(!(m < kNearGate))) {
#pragma unroll
            for (int j = 0; j < 8; j++)
                swiglu_grad<true>(xv[j], gv[j], uv[j], vg[i][j], vu[i][j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                swiglu_grad<false>(xv[j], gv[j], uv[j], vg[i][j], vu[i][j]);
        }
        __builtin_amdgcn_sched_barrier(0);   // a token's temporaries are dead before the next one's
    }
    pin(vg);
    pin(vu);
    const GradOut &dg = b.dgate, &du = b.dup;
    quant_tile<FULL, TR, true>(vg, QuantOut{dg.q_row, dg.ldq_row, dg.s_row, dg.lds_row},
                     QuantOut{dg.q_tok, dg.ldq_tok, dg.s_tok, dg.lds_tok}, p, pow2, sh);
    __syncthreads();   // the LDS tile of one gradient is read out before the other's is built
    quant_tile<FULL, TR, true>(vu, QuantOut{du.q_row, du.ldq_row, du.s_row, du.lds_row},
                     QuantOut{du.q_tok, du.ldq_tok, du.s_tok, du.lds_tok}, p, pow2, sh);
}

template <bool TR>
__global__ __launch_bounds__(TILE_THREADS) __attribute__((amdgpu_waves_per_eu(4)))
void swiglu_bwd_kernel(SwigluBwd b, int pow2)
{
    __shared__ TileShared sh;
    const auto p = place(blockIdx.y, blockIdx.x, b.tokens, b.cols);
    if (full_tile(p))
        swiglu_bwd_tile<true, TR>(b, p, pow2, sh);
    else
        swiglu_bwd_tile<false, TR>(b, p, pow2, sh);
}

dim3 tile_grid(int64_t tokens, int64_t cols)
{
    return dim3((unsigned)((cols + 127) / 128), (unsigned)((tokens + 127) / 128));
}

} // namespace

// keep_z: z is stored into the caches rather than past them, for the pass that
// reads it next (8192 x 2048: that pass 11.5 -> 9.2 us, this one 19.5 -> 20.5).
static hipError_t launch_norm_rows(const NormIn &in, uint8_t *q, int64_t ldq, float *s, bool pow2, bool keep_z,
                                   hipStream_t st)
{
    // registers for rows of 2048, 4096 and 8192 columns; two rows or more per workgroup where there
    // are many: up to 4096 workgroups of the narrow form (8192 x 2048: 21.2 us, 23.8 with 2048, 23.3
    // with 8192), up to 2048 of the others (8192 x 6144: 72.8 us, 84.8 with 1024, 77.6 with 8192)
    auto *kernel = in.cols <= 8 * NT ? norm_row_kernel<1> : in.cols <= 16 * NT ? norm_row_kernel<2> : norm_row_kernel<4>;
    const int64_t most = in.cols <= 8 * NT ? 4096 : 2048;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(in.tokens < most ? in.tokens : most)), dim3(NT), 0, st, in, q, ldq, s,
                       (in.cols + 127) / 128, (int)pow2, (int)keep_z);
    return hipGetLastError();
}

hipError_t launch_norm_act(const NormIn &in, uint8_t *q, int64_t ldq, float *s, bool pow2, hipStream_t st)
{
    return launch_norm_rows(in, q, ldq, s, pow2, false, st);
}

hipError_t launch_norm_dual(const NormIn &in, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                            int64_t ldqt, float *stok, bool pow2, hipStream_t st)
{
    const int64_t ntb = (in.tokens + 127) / 128;
    hipError_t e = launch_norm_rows(in, qr, ldqr, sr, pow2, true, st);
    if (e != hipSuccess)
        return e;
    const QuantOut to{qt, ldqt, stok, transpose_out ? ntb : in.cols};
    hipLaunchKernelGGL((transpose_out ? norm_tile_kernel<true> : norm_tile_kernel<false>),
                       tile_grid(in.tokens, in.cols), dim3(TILE_THREADS), 0, st,
                       in.res ? in.z : in.x, in.res ? in.ldz : in.ldx, in.rstd, in.w, (int)in.wbf16, in.tokens, in.cols,
                       to, (int)pow2);
    return hipGetLastError();
}

static size_t coef_bytes(int64_t tokens) { return ((size_t)tokens * 4 + 255) / 256 * 256; }

// Workgroups of the gradient's row pass: two rows each or more, so that their
// shares of dw stay small beside the rows they read, up to 512, two on every CU
// (2048 x 2048, both passes: 16.4 us, 18.1 with 1024; 8192 x 6144: 142 us,
// 147 with 1024 and 150 with 384).  Rows of up to 2048 columns leave registers for
// more workgroups on a CU: up to 1024 where each then has four rows (8192 x 2048:
// 47.3 us, and 49.5 with 512).
static int64_t bwd_groups(int64_t tokens, int64_t cols)
{
    int64_t most = 512;
    if (cols <= 8 * NT && tokens > 4 * most)
        most = tokens < 4 * 1024 ? (tokens + 3) / 4 : 1024;
    return (tokens + 1) / 2 < most ? (tokens + 1) / 2 : most;
}
static int64_t bwd_part_ld(int64_t cols) { return (cols + 15) / 16 * 16; }

size_t norm_bwd_workspace_bytes(int64_t tokens, int64_t cols)
{
    return coef_bytes(tokens) + (size_t)bwd_groups(tokens, cols) * (size_t)bwd_part_ld(cols) * 4;
}

hipError_t launch_norm_bwd(const NormBwd &b, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                           int64_t ldqt, float *stok, bool pow2, void *workspace, hipStream_t st)
{
    const int64_t nb = (b.cols + 127) / 128, ntb = (b.tokens + 127) / 128, groups = bwd_groups(b.tokens, b.cols);
    const int64_t ldp = bwd_part_ld(b.cols);
    float *coef = (float *)workspace;
    float *part = (float *)((char *)workspace + coef_bytes(b.tokens));
    if (b.tokens > 0) {
        auto *kernel = b.cols <= 8 * NT    ? norm_bwd_row_kernel<1>
                       : b.cols <= 16 * NT ? norm_bwd_row_kernel<2>
                                           : norm_bwd_row_kernel<4>;
        hipLaunchKernelGGL(kernel, dim3((unsigned)groups), dim3(NT), 0, st, b, coef, part, ldp);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    const QuantOut ro{qr, ldqr, sr, nb}, to{qt, ldqt, stok, transpose_out ? ntb : b.cols};
    hipLaunchKernelGGL((transpose_out ? norm_bwd_tile_kernel<true> : norm_bwd_tile_kernel<false>),
                       dim3(dw_groups(b.cols) + (unsigned)(nb * ntb)), dim3(TILE_THREADS), 0,
                       st, b, coef, part, (int)groups, ldp, ro, to, (int)pow2);
    return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwd &b, bool transpose_out, bool pow2, hipStream_t st)
{
    hipLaunchKernelGGL((transpose_out ? swiglu_bwd_kernel<true> : swiglu_bwd_kernel<false>),
                       tile_grid(b.tokens, b.cols), dim3(TILE_THREADS), 0, st, b, (int)pow2);
    return hipGetLastError();
}

} // namespace puro
