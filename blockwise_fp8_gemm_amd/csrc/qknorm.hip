// Norm of every query and key head and the rotation by its position, in one
// pass, and its gradient (gfx950): what stands between the joint q/k/v product
// and attention.
//
//   n = x r w, r = 1 / sqrt(mean x^2 + eps) over one head (n = x without weights)
//   y = n with its pairs (a, b) turned by theta = position * frequency:
//       m (a cos - b sin), m (b cos + a sin); elements past the rotated ones stay
//   gradient: g = dy turned back, xh = x r,
//       dx = r (w g - xh mean(w g xh)), dw = sum over tokens and heads of g xh
//
// Angles are formed in 64 bits, in turns, and reduced to half a turn either way
// before cosine and sine in FP32: a position of 2^20 has as exact a rotation as
// position 1.  Everything else is FP32.  Both directions are HBM-bound.
#include "kernels.h"
#include "tile.h"

#include <type_traits>

namespace puro {

namespace {

// Sum over each group of N lanes (8 or 16): every lane ends with the same bits.
template <int N> __device__ __forceinline__ float sum_lanes(float v)
{
    v += dpp_f<0xB1>(v);    // lane ^ 1
    v += dpp_f<0x4E>(v);    // lane ^ 2
    v += dpp_f<0x141>(v);   // 7 - lane
    if (N == 16)
        v += dpp_f<0x140>(v);   // 15 - lane
    return v;
}

// (cos, sin) of position * frequency, times m.  The frequency in turns and the
// product are off by 2^-53 of themselves each: for |position * frequency| < 2^31,
// below 2^-20 radians, and for less than 2^20, below 2^-31.  What is left of whole
// turns and quarters, at most an eighth either way, becomes an FP32 number (2^-25
// radians off at most), whose cosine and sine change places and signs by the quarter.
__device__ __forceinline__ float2 rotation(int32_t position, float frequency, float m)
{
    double turns = (double)position * ((double)frequency * 0.15915494309189533577);
    turns -= rint(turns);
    const double quarters = rint(4.0 * turns);
    float s, c;
    sincospif(2.0f * (float)(turns - 0.25 * quarters), &s, &c);
    const int n = (int)quarters;
    const float x = n & 1 ? s : c, y = n & 1 ? c : s;
    return make_float2((n + 1) & 2 ? -(x * m) : x * m, n & 2 ? -(y * m) : y * m);
}

__device__ __forceinline__ void unpack4(const uint2 &a, float v[4])
{
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
}

__device__ __forceinline__ void load4_weight(const void *w, int wbf16, int at, float v[4])
{
    if (wbf16) {
        unpack4(*reinterpret_cast<const uint2 *>((const uint16_t *)w + at), v);
    } else {
        const float4 f = *reinterpret_cast<const float4 *>((const float *)w + at);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    }
}

// Forward.  D / 8 lanes hold a head, eight elements each: in the half layout a
// rotated lane has four consecutive a and their four b (two 8-byte accesses), so
// that no pair crosses lanes.  A wave turns 512 / D heads of one token at a
// time; it forms the token's angles once, four a lane, and goes through its share
// of the heads with the next ones' loads in flight.  Bound by memory: 8192 tokens of
// 16 + 8 heads of 128, 101 MB in 19 us (5.3 TB/s; a copy reaches 5.0).
template <int D, bool INTER>
__global__ __launch_bounds__(256) void rope_kernel(RopeFwd a)
{
    constexpr int L = D / 8, HEADS = 64 / L;
    const int lane = threadIdx.x & 63, l = lane % L;
    const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6), t = wave / a.parts;
    const int part = (int)(wave % a.parts);
    if (t >= a.r.tokens)
        return;
    const int H = a.r.hq + a.r.hk, turned = a.r.rotary / 8;
    const bool rot = l < turned, half = rot && !INTER;
    const int at0 = half ? 4 * l : 8 * l, at1 = half ? a.r.rotary / 2 + 4 * l : 8 * l + 4;

    auto src = [&](int h) {
        return h < a.r.hq ? a.r.q + t * a.r.ldq + h * D : a.r.k + t * a.r.ldk + (h - a.r.hq) * D;
    };
    uint2 x0 = make_uint2(0, 0), x1 = x0;
    int h = part * HEADS + lane / L;
    if (h < H) {
        x0 = *reinterpret_cast<const uint2 *>(src(h) + at0);
        x1 = *reinterpret_cast<const uint2 *>(src(h) + at1);
    }
    float wq[8], wk[8];
    if (a.r.wq) {
        load4_weight(a.r.wq, a.r.wbf16, at0, wq);
        load4_weight(a.r.wq, a.r.wbf16, at1, wq + 4);
        load4_weight(a.r.wk, a.r.wbf16, at0, wk);
        load4_weight(a.r.wk, a.r.wbf16, at1, wk + 4);
    }
    float2 turn[4];
    if (rot) {
        const int32_t p = a.r.pos[t];
#pragma unroll
        for (int e = 0; e < 4; e++)
            turn[e] = rotation(p, a.r.freq[4 * l + e], a.r.mscale);
    }
    for (; h < H; h += a.parts * HEADS) {
        float v[8];
        unpack4(x0, v);
        unpack4(x1, v + 4);
        const int next = h + a.parts * HEADS;
        if (next < H) {
            x0 = *reinterpret_cast<const uint2 *>(src(next) + at0);
            x1 = *reinterpret_cast<const uint2 *>(src(next) + at1);
        }
        if (a.r.wq) {
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; e++)
                s = fmaf(v[e], v[e], s);
            const float r = 1.0f / sqrtf(sum_lanes<L>(s) * (1.0f / D) + a.r.eps);
            if (l == 0 && a.rstd)
                a.rstd[t * H + h] = r;
#pragma unroll
            for (int e = 0; e < 8; e++)
                v[e] = v[e] * r * (h < a.r.hq ? wq[e] : wk[e]);
        }
        if (rot) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float &p = v[INTER ? 2 * e : e], &q = v[INTER ? 2 * e + 1 : e + 4];
                const float u = p, w = q;
                p = fmaf(u, turn[e].x, -(w * turn[e].y));
                q = fmaf(w, turn[e].x, u * turn[e].y);
            }
        }
        uint16_t *dst = h < a.r.hq ? a.qo + t * a.ldqo + h * D : a.ko + t * a.ldko + (h - a.r.hq) * D;
        *reinterpret_cast<uint2 *>(dst + at0) = make_uint2(to_bf16x2(v[0], v[1]), to_bf16x2(v[2], v[3]));
        *reinterpret_cast<uint2 *>(dst + at1) = make_uint2(to_bf16x2(v[4], v[5]), to_bf16x2(v[6], v[7]));
    }
}

// ---------------------------------------------------------------------------
// Gradient.  Rotations of every token once ([token][rotary / 2], read by all the
// token's heads out of the caches), then 128 x 128 tiles of the joint gradient
// [tokens][(hq + 2 hk) D], which hold whole heads: turned back, taken through the
// norm and quantised both ways; the values' columns are quantised as they are.
// A tile's sums over its tokens of g xh go to part [token tile][column] and are
// added up in a fixed order by the last kernel.  8192 tokens, 16 + 8 + 8 heads of
// 128: 4 us, 46 us (187 MB of operands and results, 4.1 TB/s; 206 MB by the counters, of which 84 are written where codes,
// scales and shares are 70; two workgroups a CU, whose loads, shuffles and stores
// take turns, and the rotations, 64 KB a tile out of the caches) and 4 us.  A tile that
// formed its own rotations would do so once for every head, with 64-bit angles.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void rope_turn_kernel(RopeShape r, float2 *__restrict__ turn)
{
    const int half = r.rotary / 2;
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (n < r.tokens * half)
        turn[n] = rotation(r.pos[n / half], r.freq[n % half], r.mscale);
}

// How a tile's threads hold the pairs.  PAIRS: whole heads rotated in the half layout: a thread has both members of
// four pairs, in two runs.  INTER: four neighbouring pairs.  APART (part of a head in the half layout, or none of it):
// eight columns, whose other members it loads beside its own.
enum { PAIRS, INTER, APART };

template <int D, bool FULL, bool TR, int MODE, class P>
__device__ __forceinline__ void rope_bwd_tile(const RopeBwd &b, const P &p, const QuantOut &ro, const QuantOut &to,
                                              int pow2, TileShared &sh, float (*red)[128])
{
    constexpr int L = D / 8;
    const int H = b.r.hq + b.r.hk, R = b.r.rotary;
    const int64_t c0 = p.col0 + p.col(0);
    const bool in = FULL || c0 < p.cols;
    const int h = in ? (int)(c0 / D) : 0, d0 = (int)(c0 % D), up = p.col(4) - p.col(0);   // the second run's distance
    // whether the tile has query or key heads at all (the same in every lane), and this thread's columns are of one
    const bool heads = p.col0 < (int64_t)H * D, own = h < H, norm = heads && b.r.wq;
    // whether these columns are turned, in a tile that has heads; one of 128-wide heads is one head
    const bool rot = (D == 128 && MODE == PAIRS) || (own && (MODE == PAIRS || d0 < R));
    const uint16_t *dy = h < b.r.hq ? b.dq + h * D : own ? b.dk + (h - b.r.hq) * D : b.dv + (h - H) * D;
    const int64_t lddy = h < b.r.hq ? b.lddq : own ? b.lddk : b.lddv;
    const uint16_t *x = h < b.r.hq ? b.r.q + h * D : own ? b.r.k + (h - b.r.hq) * D : dy;   // not used for values
    const int64_t ldx = h < b.r.hq ? b.r.ldq : own ? b.r.ldk : lddy;
    // in the half layout the other member of a pair is R / 2 elements away
    const bool low = d0 < R / 2;
    const int other = !rot ? 0 : low ? R / 2 : -(R / 2), f0 = !rot ? 0 : MODE == INTER ? d0 / 2 : low ? d0 : d0 - R / 2;
    auto load8 = [&](const uint16_t *row) {
        if constexpr (MODE == PAIRS) {
            const uint2 a = *reinterpret_cast<const uint2 *>(row + d0), c = *reinterpret_cast<const uint2 *>(row + d0 + D / 2);
            return make_uint4(a.x, a.y, c.x, c.y);
        } else {
            return *reinterpret_cast<const uint4 *>(row + d0);
        }
    };
    // Every load comes before any arithmetic, without a branch that lanes take differently: rows past the last
    // token and columns past the last head read what is there and are left out below.
    constexpr int TURNS = MODE == APART ? 4 : 2;
    uint4 ya[RT], yb[RT], xa[RT];
    float rs[RT], w[8], dw[8], v[RT][8];
    float4 turn[RT][TURNS];
    auto load_turn = [&](int i, int64_t t) {
#pragma unroll
        for (int j = 0; j < TURNS; j++)
            turn[i][j] = *reinterpret_cast<const float4 *>(b.turn + t * (R / 2) + f0 + 2 * j);
    };
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int64_t t = FULL ? p.tk(i) : min(p.tk(i), p.tokens - 1);
        ya[i] = load8(dy + t * lddy);
        if (heads && R > 0) {
            if (MODE == APART)
                yb[i] = load8(dy + t * lddy + other);
            else
                load_turn(i, t);   // eight of them apart: there are no registers for all at once
        }
        if (norm) {
            xa[i] = load8(x + t * ldx);
            rs[i] = b.rstd[t * H + (own ? h : 0)];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        dw[j] = w[j] = 0.0f;
    if (norm) {
        const void *wp = h < b.r.hq ? b.r.wq : b.r.wk;
        load4_weight(wp, b.r.wbf16, d0, w);
        load4_weight(wp, b.r.wbf16, d0 + up, w + 4);
    }
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const bool here = in && (FULL || p.tk(i) < p.tokens);
        float g[8];
        unpack8(ya[i], g);
        if (heads && R > 0) {
            float o[8];
            if (MODE == APART) {
                unpack8(yb[i], o);
                load_turn(i, FULL ? p.tk(i) : min(p.tk(i), p.tokens - 1));
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < TURNS; j++)
#pragma unroll
                for (int e = 0; e < 2; e++) {   // rotation 2 j + e of the thread's; what is not turned keeps its bits
                    const float4 c = turn[i][j];
                    const float cs = e ? c.z : c.x, sn = e ? c.w : c.y;
                    const int n = 2 * j + e;
                    if constexpr (MODE == APART) {
                        g[n] = rot ? fmaf(g[n], cs, low ? o[n] * sn : -(o[n] * sn)) : g[n];
                    } else {
                        const int m0 = MODE == INTER ? 2 * n : n, m1 = MODE == INTER ? 2 * n + 1 : n + 4;
                        const float u = g[m0], y = g[m1];
                        g[m0] = rot ? fmaf(u, cs, y * sn) : u;
                        g[m1] = rot ? fmaf(y, cs, -(u * sn)) : y;
                    }
                }
        }
        if (norm) {
            const float r = rs[i];
            float xh[8], n[8], s = 0.0f;
            unpack8(xa[i], xh);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                xh[j] *= r;
                n[j] = g[j] * w[j];
                s = fmaf(n[j], xh[j], s);
            }
            s = sum_lanes<L>(s) * (1.0f / D);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                dw[j] = own && here ? fmaf(g[j], xh[j], dw[j]) : dw[j];
                n[j] = r * fmaf(-xh[j], s, n[j]);
                g[j] = own ? n[j] : g[j];
            }
        }
#pragma unroll
        for (int j = 0; j < 8; j++)
            v[i][j] = here ? g[j] : 0.0f;
    }
    pin(v);
    if (b.r.wq) {
        const int t = threadIdx.x, lane = t & 63;
        *reinterpret_cast<float2 *>(&red[t >> 6][p.col(first_of(lane))]) =
            cross4(dw, [](float a, float c) { return a + c; });
        __syncthreads();
        if (t < 128 && p.col0 + t < (int64_t)H * D) {
            float s = red[0][t];
#pragma unroll
            for (int k = 1; k < TileShared::WAVES; k++)
                s += red[k][t];
            b.part[(p.tok0 >> 7) * ((int64_t)H * D) + p.col0 + t] = s;
        }
    }
    if (b.dx)
        store_tile<FULL>(b.dx, b.lddx, p, v);
    quant_tile<FULL, TR, true>(v, ro, to, p, pow2, sh);
}

template <int D, bool TR, int MODE>
__global__ __launch_bounds__(TILE_THREADS) __attribute__((amdgpu_waves_per_eu(4)))
void rope_bwd_kernel(RopeBwd b, QuantOut ro, QuantOut to, int pow2)
{
    __shared__ TileShared sh;
    __shared__ float red[TileShared::WAVES][128];
    typedef typename std::conditional<MODE == PAIRS, PairPlace<D>, Place>::type P;
    // Workgroups go round the eight XCDs: eight token blocks at a time, each with all its columns on one XCD, which then
    // reads its rotations from memory once and writes row scales in whole sectors (8192 tokens: 61 -> 57 us in all).
    unsigned row = blockIdx.y, col = blockIdx.x;
    if (row < gridDim.y / 8 * 8) {
        const unsigned n = row % 8 * gridDim.x + col;
        row = row / 8 * 8 + n % 8;
        col = n / 8;
    }
    const P p = place(row, col, b.r.tokens, (int64_t)(b.r.hq + 2 * b.r.hk) * D);
    if (full_tile(p))
        rope_bwd_tile<D, true, TR, MODE>(b, p, ro, to, pow2, sh, red);
    else
        rope_bwd_tile<D, false, TR, MODE>(b, p, ro, to, pow2, sh, red);
}

// dw of 16 elements of the queries' (then the keys') weight: 64 threads each add some of the (token tile, head)
// shares, eight loads at a time, and their sums are added in a fixed order.
constexpr int DW_COLS = 16, DW_ROWS = 64;
__global__ __launch_bounds__(DW_COLS *DW_ROWS) void rope_dw_kernel(RopeBwd b, int ntb)
{
    __shared__ float red[DW_ROWS][DW_COLS];
    const int x = threadIdx.x % DW_COLS, y = threadIdx.x / DW_COLS, D = b.r.dim, per = D / DW_COLS;
    const bool keys = (int)blockIdx.x >= per;
    const int d = ((int)blockIdx.x - (keys ? per : 0)) * DW_COLS + x, heads = keys ? b.r.hk : b.r.hq, H = b.r.hq + b.r.hk;
    const float *part = b.part + (keys ? b.r.hq * D : 0) + d;
    // as many threads over the heads as fit (a power of two), the others over the tiles
    int hs = DW_ROWS;
    while (hs > heads)
        hs >>= 1;
    float s = 0.0f;
    for (int h = y & (hs - 1); h < heads; h += hs) {
#pragma unroll 8
        for (int tb = y / hs; tb < ntb; tb += DW_ROWS / hs)
            s += part[(int64_t)tb * H * D + h * D];
    }
    red[y][x] = s;
    for (int m = DW_ROWS / 2; m > 0; m >>= 1) {
        __syncthreads();
        if (y < m)
            red[y][x] += red[y + m][x];
    }
    float *dw = keys ? b.dwk : b.dwq;
    if (y == 0)
        dw[d] = b.accumulate ? dw[d] + red[0][x] : red[0][x];
}

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }
int64_t turn_count(const RopeShape &r) { return r.tokens * (r.rotary / 2); }

template <int D, bool TR, int MODE> void bwd_tiles(const RopeBwd &b, const QuantOut &ro, const QuantOut &to, int pow2, hipStream_t st)
{
    const int64_t cols = (int64_t)(b.r.hq + 2 * b.r.hk) * D;
    hipLaunchKernelGGL((rope_bwd_kernel<D, TR, MODE>), dim3((unsigned)((cols + 127) / 128), (unsigned)((b.r.tokens + 127) / 128)),
                       dim3(TILE_THREADS), 0, st, b, ro, to, pow2);
}

template <int D, bool TR> void bwd_tiles(const RopeBwd &b, const QuantOut &ro, const QuantOut &to, int pow2, hipStream_t st)
{
    if (b.r.interleaved)
        bwd_tiles<D, TR, INTER>(b, ro, to, pow2, st);
    else if (b.r.rotary == D)
        bwd_tiles<D, TR, PAIRS>(b, ro, to, pow2, st);
    else
        bwd_tiles<D, TR, APART>(b, ro, to, pow2, st);
}

} // namespace

hipError_t launch_rope(RopeFwd a, hipStream_t st)
{
    // A token's heads over several waves where tokens are few: up to 4096 waves (four a SIMD), each of which forms the
    // token's angles again.  24 heads of 128: 256 tokens 4.2 us, a wave for each 6.3; 2048 tokens 8.9, spread out 12.2.
    const int passes = (a.r.hq + a.r.hk + 512 / a.r.dim - 1) / (512 / a.r.dim);
    const int64_t want = a.r.tokens ? 4096 / a.r.tokens : 1;
    a.parts = (int)(want < 1 ? 1 : want < passes ? want : passes);
    const unsigned grid = (unsigned)((a.r.tokens * a.parts + 3) / 4);
    auto *kernel = a.r.dim == 64 ? (a.r.interleaved ? rope_kernel<64, true> : rope_kernel<64, false>)
                                 : (a.r.interleaved ? rope_kernel<128, true> : rope_kernel<128, false>);
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

size_t rope_bwd_workspace_bytes(const RopeShape &r, bool norm)
{
    const int64_t ntb = (r.tokens + 127) / 128;
    return pad256((size_t)turn_count(r) * sizeof(float2)) +
           (norm ? pad256((size_t)ntb * (size_t)(r.hq + r.hk) * (size_t)r.dim * 4) : 0);
}

hipError_t launch_rope_bwd(RopeBwd b, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt, int64_t ldqt,
                           float *stok, bool pow2, void *workspace, hipStream_t st)
{
    const int64_t turns = turn_count(b.r), ntb = (b.r.tokens + 127) / 128;
    const int64_t cols = (int64_t)(b.r.hq + 2 * b.r.hk) * b.r.dim;
    float2 *turn = (float2 *)workspace;
    b.turn = turn;
    b.part = (float *)((char *)workspace + pad256((size_t)turns * sizeof(float2)));
    hipError_t e = hipSuccess;
    if (turns > 0) {
        hipLaunchKernelGGL(rope_turn_kernel, dim3((unsigned)((turns + 255) / 256)), dim3(256), 0, st, b.r, turn);
        e = hipGetLastError();
    }
    if (e == hipSuccess && b.r.tokens > 0) {
        const QuantOut ro{qr, ldqr, sr, (cols + 127) / 128}, to{qt, ldqt, stok, transpose_out ? ntb : cols};
        if (b.r.dim == 64)
            transpose_out ? bwd_tiles<64, true>(b, ro, to, pow2, st) : bwd_tiles<64, false>(b, ro, to, pow2, st);
        else
            transpose_out ? bwd_tiles<128, true>(b, ro, to, pow2, st) : bwd_tiles<128, false>(b, ro, to, pow2, st);
        e = hipGetLastError();
    }
    if (e == hipSuccess && b.r.wq) {
        hipLaunchKernelGGL(rope_dw_kernel, dim3((unsigned)(2 * b.r.dim / DW_COLS)), dim3(DW_COLS * DW_ROWS), 0,
                           st, b, (int)ntb);
        e = hipGetLastError();
    }
    return e;
}

} // namespace puro
