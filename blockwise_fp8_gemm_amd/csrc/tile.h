// What the kernels that form FP32 values and quantise them in place share (gfx950): a 128-token x
// 128-column tile's loads, stores and both quantisations, and the reductions within a wave.
#pragma once

#include "common.h"
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
    static constexpr bool SPLIT = false;
    int64_t tok0, col0, tokens, cols;
    int cc, rq;
    __device__ __forceinline__ int col(int j) const { return 8 * cc + j; }   // column j of the thread's eight, in the tile
    __device__ __forceinline__ int64_t tk(int i) const { return tok0 + RT * rq + i; }
    __device__ __forceinline__ int64_t c0() const { return col0 + 8 * cc; }
};
// The same with a thread's columns in two runs of four, which are the two members of four pairs (j, j + D / 2) of a
// head of D.
template <int D> struct PairPlace : Place {
    static constexpr bool SPLIT = true;
    __device__ __forceinline__ PairPlace(const Place &p) : Place(p) {}
    __device__ __forceinline__ int low() const { return D == 128 ? 4 * cc : 64 * (cc >> 3) + 4 * (cc & 7); }
    __device__ __forceinline__ int col(int j) const { return low() + (j < 4 ? j : D / 2 + j - 4); }
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

// A thread's eight codes of one token, at `row` (the tensor's).
template <bool FULL, class P> __device__ __forceinline__ void store_codes(uint8_t *row, const P &p, uint32_t lo, uint32_t hi)
{
    if constexpr (P::SPLIT) {   // whole heads lie inside or outside the tensor
        if (FULL || p.col0 + p.col(0) < p.cols) {
            __builtin_nontemporal_store(lo, reinterpret_cast<uint32_t *>(row + p.col0 + p.col(0)));
            __builtin_nontemporal_store(hi, reinterpret_cast<uint32_t *>(row + p.col0 + p.col(4)));
        }
    } else if (FULL) {
        store_nt(row + p.c0(), lo, hi);
    } else {
        store8_codes(row, p.c0(), p.cols, lo, hi);
    }
}

template <bool SLOW, bool FULL, bool TR, bool ROWS, class P>
__device__ __forceinline__ void tile_codes(const float (&v)[RT][8], const Scale &own, const QuantOut &ro,
                                           const QuantOut &to, const P &p, TileShared &sh)
{
    if constexpr (ROWS) {
        const Scale sr[RT] = {row_scale<0>(own), row_scale<1>(own), row_scale<2>(own), row_scale<3>(own)};
        uint8_t *qr = ro.q + p.tk(0) * ro.ldq;
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const uint32_t lo = codes4<SLOW>(v[i][0], v[i][1], v[i][2], v[i][3], sr[i]);
            const uint32_t hi = codes4<SLOW>(v[i][4], v[i][5], v[i][6], v[i][7], sr[i]);
            if (FULL || p.tk(i) < p.tokens)
                store_codes<FULL>(qr + i * ro.ldq, p, lo, hi);
        }
    }
    uint32_t word[8];   // RT codes of a column, a byte each
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const Scale c{SLOW ? sh.scl[p.col(j)] : 0.0f, sh.rcl[p.col(j)], sh.rll[p.col(j)]};
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
                store_codes<false>(to.q + p.tk(i) * to.ldq, p, lo, hi);
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        *reinterpret_cast<uint32_t *>(&sh.tile[p.col(j)][RT * p.rq]) = word[j];
}

template <bool FULL, bool TR, bool ROWS, class P>
__device__ __forceinline__ void quant_tile(const float (&v)[RT][8], const QuantOut &ro, const QuantOut &to,
                                           const P &p, int pow2, TileShared &sh)
{
    constexpr int WAVES = TileShared::WAVES;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t bx = p.col0 >> 7, by = p.tok0 >> 7;

    float m[8];
#pragma unroll
    for (int j = 0; j < 8; j++)
        m[j] = absmax3(v[2][j], v[3][j], absmax3(v[0][j], v[1][j], 0.0f));
    *reinterpret_cast<float2 *>(&sh.red[wave][p.col(first_of(lane))]) =
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

template <bool FULL, class P>
__device__ __forceinline__ void store_tile(uint16_t *x, int64_t ldx, const P &p, const float (&v)[RT][8])
{
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const uint32_t o[4] = {to_bf16x2(v[i][0], v[i][1]), to_bf16x2(v[i][2], v[i][3]), to_bf16x2(v[i][4], v[i][5]),
                               to_bf16x2(v[i][6], v[i][7])};
        uint16_t *row = x + p.tk(i) * ldx;
        if constexpr (P::SPLIT) {
            if (FULL || (p.tk(i) < p.tokens && p.col0 + p.col(0) < p.cols)) {
                store_nt(row + p.col0 + p.col(0), o[0], o[1]);
                store_nt(row + p.col0 + p.col(4), o[2], o[3]);
            }
        } else if (FULL) {
            store_nt(row + p.c0(), o[0], o[1], o[2], o[3]);
        } else if (p.tk(i) < p.tokens) {
            store8_bf16(row, p.c0(), p.cols, o);
        }
    }
}

// Whole tiles (uniform over the workgroup) and edge tiles are two bodies of one kernel.
__device__ __forceinline__ bool full_tile(const Place &p)
{
    return p.tok0 + 128 <= p.tokens && p.col0 + 128 <= p.cols;
}

} // namespace

} // namespace puro
