// Attention of packed sequences with grouped heads, and its gradient (gfx950).
//
//   S = c q k^T,  L = log sum exp S,  P = exp(S - L),  o = P v
//   dP = do v^T,  dS = P (dP - D),  D = sum over the head of do o
//   dv = P^T do,  dq = c dS k,  dk = c dS^T q
//
// Query i of n sees keys 0 .. m - 1, or those of them up to i + m - n with a causal mask.
// Products run on the BF16 matrix cores (32x32x16) with FP32 accumulation.
// Every operand tile is a [rows][D] run of BF16 rows in LDS, copied there
// straight from memory, and read in two ways: rows (a lane takes 8 consecutive
// elements of one row) and columns (transposing reads).  Scores are formed
// transposed where the softmax runs along the keys (a lane then owns one query,
// so that maximum, sum and rescaling are per lane), and an accumulator's 16
// values of a lane are, in order, what the next product wants as its operand:
// the order of a product's contraction is free, so that the transposing reads
// take their rows in the accumulator's order instead of moving P between lanes.
//
// P and dS enter their products as BF16 numbers (each rounded once, 2^-8 of
// itself; the results are BF16 too, and the roundings of a row's many terms
// average out); scores, statistics and every sum are FP32.
#include "common.h"
#include "kernels.h"

#include <type_traits>

namespace puro {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr float kNoMax = -0x1p100f;   // running maximum (log2 units) before the first visible key
constexpr float kLog2e = 0x1.715476p0f, kLn2 = 0x1.62e430p-1f;

__device__ __forceinline__ uint32_t lds_addr(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// 16 (4) bytes per lane from base + off (base wave-uniform) to the wave's LDS
// base + 16 (4) lane.  M0 is set in the same statement and nothing else here
// reads it; the copies count in vmcnt, which wait_copies() waits on.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(const void *base, uint32_t off, uint8_t *lds_wave_base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(lds_addr(lds_wave_base)) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const void *base, uint32_t off, void *lds_wave_base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
                 :: "v"(off), "s"(base), "s"(lds_addr(lds_wave_base)) : "memory", "m0");
}
#pragma clang diagnostic pop
template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// ---------------------------------------------------------------------------
// Tiles of BF16 rows in LDS.  A tile is made of 1 KB pieces of 1024 / ROW rows,
// each filled by one copy of a wave (lane l's 16 bytes at 16 l) and followed by a
// little padding.  Within a piece, segment 4 x + y (16 bytes) of row r lies at
// 256 x + 64 (r % 4) + 16 y; with heads of 64 rows r % 8 >= 4 follow 512 bytes
// behind, their y with the low bit flipped.  So 16 consecutive rows hold one
// segment on 16 different places of the 256 bytes that the banks span (row
// reads), and a transposing read's four rows x 64 bytes lie side by side; and
// both addresses are one register a lane plus constants.
// ---------------------------------------------------------------------------
template <int D> struct Tile {
    static constexpr int SEGS = D / 8, SLICES = D / 16, BLOCKS = D / 32;
    static constexpr int PIECE = 64 / SEGS;                       // rows of a piece: 4 or 8
    static constexpr int STRIDE = 1024 + (D == 128 ? 16 : 32);    // bytes from piece to piece
    static constexpr int bytes(int rows) { return rows / PIECE * STRIDE; }

    // A wave's share of tiles of ROWS rows: the lane's offsets from the first row, of row stride ld bytes.
    template <int ROWS, int NW> struct Stage {
        static constexpr int N = ROWS / PIECE / NW;
        static_assert(ROWS / PIECE % NW == 0, "whole pieces per wave");
        uint32_t ld, off[N];
        int row, seg;

        __device__ __forceinline__ Stage(int64_t stride, int wave, int lane) : ld((uint32_t)stride * 2)
        {
            const int sub = D == 128 ? 0 : lane >> 5, x = D == 128 ? lane >> 4 : (lane >> 4) & 1;
            row = PIECE * wave + 4 * sub + ((lane >> 2) & 3);
            seg = (4 * x + ((lane & 3) ^ sub)) * 16;
#pragma unroll
            for (int i = 0; i < N; i++)
                off[i] = (uint32_t)(row + PIECE * NW * i) * ld + (uint32_t)seg;
        }

        // The tile that begins at g to t.  Rows past `last` are copies of it, so that nothing behind a
        // sequence is read.
        __device__ __forceinline__ void operator()(uint8_t *t, const uint16_t *g, int last, int wave) const
        {
            if (last >= ROWS - 1) {
#pragma unroll
                for (int i = 0; i < N; i++)
                    copy16(g, off[i], t + (wave + NW * i) * STRIDE);
            } else {
#pragma unroll
                for (int i = 0; i < N; i++)
                    copy16(g, (uint32_t)min(row + PIECE * NW * i, last) * ld + (uint32_t)seg, t + (wave + NW * i) * STRIDE);
            }
        }
    };

    // Where the lane's part of a row read and of a column read begins.
    __device__ __forceinline__ static int row_base(int lane)
    {
        const int r = lane & 31, h = lane >> 5;
        return D == 128 ? (r >> 2) * STRIDE + (r & 3) * 64 + h * 16
                        : (r >> 3) * STRIDE + ((r >> 2) & 1) * 512 + (r & 3) * 64 + ((h ^ (r >> 2)) & 1) * 16;
    }
    __device__ __forceinline__ static int col_base(int lane)
    {
        const int h = lane >> 5, i = lane & 15, y = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
        return D == 128 ? h * STRIDE + (i >> 2) * 64 + y * 16 + 8 * (i & 1)
                        : h * 512 + (i >> 2) * 64 + (y ^ h) * 16 + 8 * (i & 1);
    }

    // Rows row0 + lane % 32 (row0 a multiple of 32), elements 16 s + 8 (lane / 32) .. +7; t: the tile plus row_base.
    __device__ __forceinline__ static v8bf rows(const uint8_t *t, int row0, int s)
    {
        return __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u *>(
                                            t + row0 / PIECE * STRIDE + (s >> 1) * 256 + (s & 1) * 32));
    }

    // Column 32 b + lane % 32 of the 16 rows from row0 on (a multiple of 16): rows 4 h .. 4 h + 3 and
    // 8 + 4 h .. 8 + 4 h + 3, h = lane / 32, which is the order of an accumulator's 8 values; t: the tile plus
    // col_base.
    __device__ __forceinline__ static v8bf cols(const uint8_t *t, int row0, int b)
    {
        typedef __attribute__((address_space(3))) v4s lds_v4s;
        v4s q[2];
#pragma unroll
        for (int j = 0; j < 2; j++)
            q[j] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(t + (row0 + 8 * j) / PIECE * STRIDE + b * 256));
        return __builtin_bit_cast(v8bf, __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }

    // Row `row`'s elements for rows()'s place in a product, straight from memory.
    __device__ __forceinline__ static void load(const uint16_t *row, int lane, v8bf (&f)[SLICES])
    {
#pragma unroll
        for (int s = 0; s < SLICES; s++)
            f[s] = __builtin_bit_cast(v8bf, *reinterpret_cast<const v4u *>(row + 16 * s + 8 * (lane >> 5)));
    }
};

__device__ __forceinline__ v16f mfma(v8bf a, v8bf b, v16f c) { return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0); }

__device__ __forceinline__ v16f splat(float x) { return v16f{x, x, x, x, x, x, x, x, x, x, x, x, x, x, x, x}; }

// Row of an accumulator's value i in this lane.
__device__ __forceinline__ int acc_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// f(0) .. f(N - 1) with constant arguments.
template <int N, class F> __device__ __forceinline__ void each(F f)
{
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// N products: use(i, load(i)) in order, with the next AHEAD operands' reads from LDS in flight.  The scheduling
// barriers hold every read at its place: left alone the compiler puts each in front of its product, which then
// waits for it.  The first reads may be made earlier, by first().
template <int N, int AHEAD = 6, class T = v8bf> struct Feed {
    static constexpr int RING = N < AHEAD ? N : AHEAD;
    T f[RING];

    template <class L> __device__ __forceinline__ void first(L load)
    {
        each<RING>([&](auto I) { f[I] = load(I); });
    }
    template <class L, class U> __device__ __forceinline__ void run(L load, U use)
    {
        each<N>([&](auto I) {
            constexpr int i = decltype(I)::value;
            __builtin_amdgcn_sched_barrier(0);
            use(I, f[i % RING]);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (i + RING < N)
                f[i % RING] = load(std::integral_constant<int, i + RING>{});
        });
    }
};
template <int N, class L, class U> __device__ __forceinline__ void feed(L load, U use)
{
    Feed<N> f;
    f.first(load);
    f.run(load, use);
}

// Holds an operand in registers from here on, its load from memory waited for.
template <int N> __device__ __forceinline__ void pin(v8bf (&f)[N])
{
#pragma unroll
    for (int i = 0; i < N; i++) {
        v4u w = __builtin_bit_cast(v4u, f[i]);
        asm volatile("" : "+v"(w));
        f[i] = __builtin_bit_cast(v8bf, w);
    }
}

// Values 8 s .. 8 s + 7 of an accumulator as an operand.
__device__ __forceinline__ v8bf operand(const v16f &v, int s)
{
    const v4u w = {to_bf16x2(v[8 * s], v[8 * s + 1]), to_bf16x2(v[8 * s + 2], v[8 * s + 3]),
                   to_bf16x2(v[8 * s + 4], v[8 * s + 5]), to_bf16x2(v[8 * s + 6], v[8 * s + 7])};
    return __builtin_bit_cast(v8bf, w);
}

// x of the lane's other half (lane ^ 32).
__device__ __forceinline__ float other_half(float x)
{
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// A sequence's rows, held inside the tensor and the announced maximum whatever the arrays say (none where it starts before
// row 0), and how many the arrays give it (up to 2^30).
struct Rows {
    int start, len, whole;
};
__device__ __forceinline__ Rows rows_of(const int32_t *off, const int32_t *len, int s, int64_t tokens, int most)
{
    const int64_t total = tokens, a = off[s];
    const int64_t start = a < 0 || a > total ? total : a;
    int64_t n = len ? (int64_t)len[s] : (int64_t)off[s + 1] - a;
    n = n < 0 ? 0 : n < 1 << 30 ? n : 1 << 30;
    const int whole = (int)n;
    n = n < total - start ? n : total - start;
    n = n < most ? n : most;
    return Rows{(int)start, (int)n, whole};
}
__device__ __forceinline__ Rows uniform(const Rows &r) { return Rows{uniform(r.start), uniform(r.len), uniform(r.whole)}; }
__device__ __forceinline__ Rows q_rows(const AttnShape &a, int s) { return rows_of(a.q_off, a.q_len, s, a.tokens_q, a.max_q); }
__device__ __forceinline__ Rows k_rows(const AttnShape &a, int s) { return rows_of(a.k_off, a.k_len, s, a.tokens_k, a.max_k); }

// Causal: query i sees the keys up to i + shift.  By the whole sequences, so that rows that are kept see no other keys
// when rows behind them are left out.
__device__ __forceinline__ int shift_of(const Rows &q, const Rows &k) { return k.whole - q.whole; }

// A lane's 4 D / 32 runs of four values of one row (acc_row's order), times f, as BF16.
template <int D> __device__ __forceinline__ void store_row(uint16_t *row, const v16f (&acc)[D / 32], float f, int lane)
{
#pragma unroll
    for (int b = 0; b < D / 32; b++)
#pragma unroll
        for (int g = 0; g < 4; g++)
            *reinterpret_cast<uint2 *>(row + 32 * b + 8 * g + 4 * (lane >> 5)) =
                make_uint2(to_bf16x2(acc[b][4 * g] * f, acc[b][4 * g + 1] * f),
                           to_bf16x2(acc[b][4 * g + 2] * f, acc[b][4 * g + 3] * f));
}

// ---------------------------------------------------------------------------
// Forward.  Running state of 32 queries of a wave (one per lane and half):
// maximum m in log2 units, this half's share of the sum, the transposed output.
// The maximum only moves, and sum and output are only rescaled, when a score
// passes it by more than 8 (2^8), or with heads of 128 when the sum of a lane's
// scores of a tile does: P stays below 2^8 and keeps its relative precision, and
// most tiles need no rescaling.
// ---------------------------------------------------------------------------
template <int D> struct Softmax {
    float m = kNoMax, l = 0.0f;
    v16f o[D / 32];

    __device__ __forceinline__ Softmax()
    {
#pragma unroll
        for (int b = 0; b < D / 32; b++)
            o[b] = splat(0.0f);
    }

    // The matrix cores' part: ADD: the P v of the last N blocks of 32 keys (tile rows vt); NEW: the scores,
    // transposed, of the next ones (tile rows kt).
    template <int N, bool ADD, bool NEW>
    __device__ __forceinline__ void products(const uint8_t *vt, const v8bf (&p)[2 * N], const uint8_t *kt,
                                             const v8bf (&q)[D / 16], v16f (&s)[N], int lane)
    {
        constexpr int B = D / 32, A = ADD ? 2 * N * B : 0, T = A + (NEW ? N * D / 16 : 0);
        const uint8_t *kr = kt + Tile<D>::row_base(lane), *vc = vt + Tile<D>::col_base(lane);
        if (NEW) {
#pragma unroll
            for (int n = 0; n < N; n++)
                s[n] = splat(0.0f);
        }
        feed<T>(
            [&](auto I) {
                constexpr int i = decltype(I)::value;
                if constexpr (i < A)
                    return Tile<D>::cols(vc, 16 * (i / B), i % B);
                else
                    return Tile<D>::rows(kr, 32 * ((i - A) % N), (i - A) / N);
            },
            [&](auto I, const v8bf &f) {
                constexpr int i = decltype(I)::value;
                if constexpr (i < A)
                    o[i % B] = mfma(f, p[i / B], o[i % B]);
                else
                    s[(i - A) % N] = mfma(f, q[(i - A) / N], s[(i - A) % N]);
            });
    }

    // 2^(c2 s - m) as the next product's operand, and their sum over the lane.
    template <int N> __device__ __forceinline__ float exponentials(const v16f (&s)[N], v8bf (&p)[2 * N], float c2) const
    {
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
            for (int k = 0; k < 2; k++) {
                float e[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    e[i] = __builtin_amdgcn_exp2f(fmaf(s[n][8 * k + i], c2, -m));
                    sum += e[i];
                }
                const v4u w = {to_bf16x2(e[0], e[1]), to_bf16x2(e[2], e[3]), to_bf16x2(e[4], e[5]), to_bf16x2(e[6], e[7])};
                p[2 * n + k] = __builtin_bit_cast(v8bf, w);
            }
        return sum;
    }

    // The running maximum up to the scores, where one lies more than 2^SLACK above it.
    template <int N, int SLACK> __device__ __forceinline__ void raise(const v16f (&s)[N], float c2)
    {
        float top = s[0][0];
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
            for (int i = 0; i < 16; i++)
                top = fmaxf(top, s[n][i]);
        top = fmaxf(top, other_half(top)) * c2;
        if (__any(top > m + (float)SLACK)) {
            const float now = fmaxf(m, top), f = __builtin_amdgcn_exp2f(m - now);
            m = now;
            l *= f;
#pragma unroll
            for (int b = 0; b < D / 32; b++)
                o[b] *= f;
        }
    }

    // P of the blocks, and their share of the sum.  first: the blocks' first key; start: that of all of them; lim: the
    // lane's last visible key; masked: whether some key of the blocks may be hidden.  With heads of 128 the maximum is
    // looked for only among the first keys and where P's sum shows that scores have left it behind (2 x 4096 causal
    // 125 us, and 127.5 with a search in every tile; heads of 64: 82 and 80.5).  It then goes up to the highest of them, so
    // that a sum is at most the number of its keys again: with 2^8 left between them, many scores a little below that
    // would have every later tile searched and formed twice.
    template <int N>
    __device__ __forceinline__ void weigh(v16f (&s)[N], v8bf (&p)[2 * N], float c2, int first, int start, int lim, bool masked,
                                          int lane)
    {
        if (masked) {
#pragma unroll
            for (int n = 0; n < N; n++)
#pragma unroll
                for (int i = 0; i < 16; i++)
                    s[n][i] = first + 32 * n + acc_row(i, lane) > lim ? -INFINITY : s[n][i];
        }
        float sum = INFINITY;
        if (D == 128 && first != start)
            sum = exponentials<N>(s, p, c2);
        if (D != 128 || __any(!(sum <= 256.0f))) {
            raise<N, D == 128 ? 0 : 8>(s, c2);
            sum = exponentials<N>(s, p, c2);
        }
        l += sum;
        pin(p);   // formed here, not where the products want them
    }
};

// Share `split` of n tiles (at most 2^18: of 32 keys, of 2^23; in at most 2^7 shares).
__device__ __forceinline__ int share(int n, int split, int splits) { return uniform(n * split / splits); }

// 1 / l of a row's sum, and its lse.  0 is a row that sees nothing; NaN stays NaN.
__device__ __forceinline__ float reciprocal(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float log_sum(float m, float l) { return l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2; }

// Where row t's partial results of a split go: [split][head][row].
__device__ __forceinline__ int64_t part_row(const AttnFwd &a, int split, int head, int t)
{
    return ((int64_t)split * a.s.hq + head) * a.s.tokens_q + t;
}

// The results of one query row, whole or a split's share.
template <int D>
__device__ __forceinline__ void put_row(const AttnFwd &a, Softmax<D> &x, int split, int head, int t, int lane)
{
    const float l = x.l + other_half(x.l);
    if (a.splits == 1) {
        store_row<D>(a.o + (int64_t)t * a.ldo + head * D, x.o, reciprocal(l), lane);
        if (a.lse && lane < 32)
            a.lse[(int64_t)head * a.s.tokens_q + t] = log_sum(x.m, l);
        return;
    }
    const int64_t p = part_row(a, split, head, t);
    float *o = a.part + p * D;
#pragma unroll
    for (int b = 0; b < D / 32; b++)
#pragma unroll
        for (int g = 0; g < 4; g++)
            *reinterpret_cast<float4 *>(o + 32 * b + 8 * g + 4 * (lane >> 5)) =
                make_float4(x.o[b][4 * g], x.o[b][4 * g + 1], x.o[b][4 * g + 2], x.o[b][4 * g + 3]);
    if (lane < 32)
        a.stat[p] = make_float2(x.m, l);
}

// Many rows: NW waves of 32 rows, a query of one head each, HV times; 64 keys (128 of narrow heads) at a time through
// LDS.  The HV waves of the same rows take every HV-th tile, and their results meet at the end.  Bound by the matrix
// cores and the exponentials, which hardly overlap: 2 x 4096 causal queries, 16 heads of 128, 137 GFLOP in 125 us (1.1
// PFLOP/s), matrix cores busy 0.6 of the time, no bank conflicts, 82 MB fetched.  128 keys a tile with heads of 128 took
// 177 us against 132, 64 keys with heads of 64 37 against 29.5 (packed lengths of 1 to 1500).
template <int D, int NW, int HV>
__global__ __launch_bounds__(64 * NW * HV, 2) void attn_fwd_kernel(AttnFwd a)
{
    constexpr int R = 32 * NW, KT = 8192 / D, TILE = Tile<D>::bytes(KT), N = KT / 32;
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][HV][TILE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % NW, part = wave / NW;
    // blocks of later rows, which see more keys, first; a sequence's key head on one XCD where their
    // number is a multiple of 8 (workgroups go round the XCDs).  The query heads of a key head share its tiles.
    const int units = a.s.seqs * a.s.hk, group = a.s.hq / a.s.hk;
    const int x = uniform((int)blockIdx.x / units), unit = (int)blockIdx.x - x * units;
    const int seq = uniform(unit / a.s.hk), kh = unit - seq * a.s.hk;
    const int later = uniform(x / a.splits), split = x - later * a.splits, r0 = (a.blocks - 1 - later) * R;
    const Rows q = uniform(q_rows(a.s, seq)), k = uniform(k_rows(a.s, seq));
    const int rows = q.len * group;   // (query, head) pairs, a query's heads side by side
    if (r0 >= rows)
        return;
    const int shift = shift_of(q, k), last = uniform((min(r0 + R, rows) - 1) / group);
    const int seen = a.s.causal ? max(0, min(k.len, last + 1 + shift)) : k.len;
    const int tiles = (seen + KT - 1) / KT, t0 = share(tiles, split, a.splits), t1 = share(tiles, split + 1, a.splits);
    const int rounds = (t1 - t0 + HV - 1) / HV;

    const uint16_t *kp = a.k + (int64_t)k.start * a.ldk + kh * D, *vp = a.v + (int64_t)k.start * a.ldv + kh * D;
    const typename Tile<D>::template Stage<KT, NW * HV> copy_k(a.ldk, wave, lane), copy_v(a.ldv, wave, lane);
    // a round's tiles; places past the last tile hold it again, and its keys are hidden there
    auto stage_k = [&](int n) {
        if (n < rounds)
#pragma unroll
            for (int h = 0; h < HV; h++) {
                const int j = min(t0 + HV * n + h, t1 - 1) * KT;
                copy_k(lds[0][n & 1][h], kp + (int64_t)j * a.ldk, k.len - 1 - j, wave);
            }
    };
    auto stage_v = [&](int n) {
        if (n < rounds)
#pragma unroll
            for (int h = 0; h < HV; h++) {
                const int j = min(t0 + HV * n + h, t1 - 1) * KT;
                copy_v(lds[1][n & 1][h], vp + (int64_t)j * a.ldv, k.len - 1 - j, wave);
            }
    };
    // everyone's copies of round n's K tiles and the last one's V tiles have landed and the places of the ones before
    // are free
    auto turn = [&](int n) {
        wait_copies<0>();
        __builtin_amdgcn_sched_barrier(0);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        stage_k(n + 1);
        stage_v(n);
    };
    stage_k(0);
    const int w0 = r0 + 32 * rw, r = w0 + (lane & 31), rc = min(r, rows - 1);
    const int i = rc / group, head = kh * group + (rc - i * group), row = q.start + i;
    v8bf qf[D / 16];
    Tile<D>::load(a.q + (int64_t)row * a.ldq + head * D, lane, qf);
    const int lim = min(t1 * KT - 1, a.s.causal ? min(k.len - 1, i + shift) : k.len - 1);
    // the wave's first row's
    const int low = min(t1 * KT - 1, a.s.causal ? min(k.len - 1, uniform(w0 / group) + shift) : k.len - 1);

    // Between two barriers a wave has the matrix cores' part of a tile (the last one's P v, the next scores) and
    // the exponentials of one: the early half of the waves in that order, the late half, which is on the same
    // SIMDs, the other way round, so that one's products run beside the other's exponentials.
    const bool late = wave >= NW * HV / 2;
    Softmax<D> st;
    v16f s[N];
    v8bf p[2 * N];
    pin(qf);
    if (rounds > 0) {
        auto weigh = [&](int n) {
            const int j = (t0 + HV * n + part) * KT;
            st.template weigh<N>(s, p, a.c2, j, (t0 + part) * KT, lim, j + KT - 1 > low, lane);
        };
        turn(0);
        st.template products<N, false, true>(lds[1][0][part], p, lds[0][0][part], qf, s, lane);
        for (int n = 0; n < rounds - 1; n++) {
            if (late)
                turn(n + 1);
            weigh(n);
            if (!late)
                turn(n + 1);
            st.template products<N, true, true>(lds[1][n & 1][part], p, lds[0][(n + 1) & 1][part], qf, s, lane);
        }
        if (late)
            turn(rounds);
        weigh(rounds - 1);
        if (!late)
            turn(rounds);
        st.template products<N, true, false>(lds[1][(rounds - 1) & 1][part], p, lds[0][0][part], qf, s, lane);
    }
    if constexpr (HV == 2) {
        constexpr int V = D / 2;   // a lane's values of o
        static_assert(NW * (V + 2) * 256 <= (int)sizeof(lds), "a half's results take the tiles' place");
        float *x = reinterpret_cast<float *>(lds) + rw * (V + 2) * 64 + lane;
        __syncthreads();
        if (part == 1) {
#pragma unroll
            for (int e = 0; e < V; e++)
                x[e * 64] = st.o[e / 16][e % 16];
            x[V * 64] = st.m;
            x[(V + 1) * 64] = st.l;
        }
        __syncthreads();
        if (part == 1)
            return;
        const float m = fmaxf(st.m, x[V * 64]);
        const float f = __builtin_amdgcn_exp2f(st.m - m), g = __builtin_amdgcn_exp2f(x[V * 64] - m);
        st.m = m;
        st.l = fmaf(g, x[(V + 1) * 64], f * st.l);
#pragma unroll
        for (int e = 0; e < V; e++)
            st.o[e / 16][e % 16] = fmaf(g, x[e * 64], f * st.o[e / 16][e % 16]);
    }
    if (r < rows)
        put_row<D>(a, st, split, head, row, lane);
}

// Few rows (at most 32 of a key head's queries over all its query heads): a wave
// holds them all and the workgroup's two waves take keys of their own, 32 at a
// time through LDS of their own; their results are added up at the end.  Bound by
// reading the keys and values once: 16 sequences of up to 16384 keys, 500 MB in 101 us
// (4.9 TB/s; a copy reaches 5.0).  Two waves a workgroup let every wave go on
// without a barrier; four, without the heads changing places, took 123.5 us against 113.
constexpr int ROW_WAVES = 2;
template <int D>
__global__ __launch_bounds__(64 * ROW_WAVES) void attn_rows_kernel(AttnFwd a)
{
    constexpr int NW = ROW_WAVES, KW = 32, TILE = Tile<D>::bytes(KW), S = 2, WAVE = S * 2 * TILE;
    static_assert(WAVE >= 32 * (D + 4) * 4, "a wave's results take its tiles' place");
    __shared__ __attribute__((aligned(16))) uint8_t lds[NW][WAVE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int units = a.s.seqs * a.s.hk, group = a.s.hq / a.s.hk;
    // heads change places from sequence to sequence and share to share: with as many as XCDs each would read one
    // head's 256 bytes of every row
    const int split = uniform((int)blockIdx.x / units), unit = (int)blockIdx.x - split * units;
    const int seq = uniform(unit / a.s.hk), kh = uniform((unit - seq * a.s.hk + seq + split) % a.s.hk);
    const Rows q = uniform(q_rows(a.s, seq)), k = uniform(k_rows(a.s, seq));
    const int cols = q.len * group;
    if (cols == 0)
        return;
    const int shift = shift_of(q, k), seen = k.len;
    const int tiles = (seen + KW - 1) / KW, parts = a.splits * NW, part = split * NW + wave;
    const int t0 = share(tiles, part, parts), t1 = share(tiles, part + 1, parts);

    const uint16_t *kp = a.k + (int64_t)k.start * a.ldk + kh * D, *vp = a.v + (int64_t)k.start * a.ldv + kh * D;
    const typename Tile<D>::template Stage<KW, 1> copy_k(a.ldk, 0, lane), copy_v(a.ldv, 0, lane);
    uint8_t *const kt = lds[wave], *const vt = lds[wave] + 2 * TILE;
    auto stage_k = [&](int t) {
        if (t < t1)
            copy_k(kt + (t & 1) * TILE, kp + (int64_t)t * KW * a.ldk, k.len - 1 - t * KW, 0);
    };
    auto stage_v = [&](int t) {
        if (t < t1)
            copy_v(vt + (t & 1) * TILE, vp + (int64_t)t * KW * a.ldv, k.len - 1 - t * KW, 0);
    };
    stage_k(t0);
    stage_v(t0);
    stage_k(t0 + 1);
    stage_v(t0 + 1);
    const int c = min(lane & 31, cols - 1), i = c / group, head = kh * group + c % group;
    v8bf qf[D / 16];
    Tile<D>::load(a.q + (int64_t)(q.start + i) * a.ldq + head * D, lane, qf);
    const int lim = a.s.causal ? min(k.len - 1, i + shift) : k.len - 1;
    const int low = a.s.causal ? min(k.len - 1, shift) : k.len - 1;
    pin(qf);

    // A tile's place is filled again as soon as it is read: of a wave's four tiles in LDS three or more are on
    // their way at any time.  (Two of four: 4.2 TB/s of keys and values.)
    constexpr int C = KW / Tile<D>::PIECE;   // copies of a tile
    Softmax<D> st;
    for (int t = t0; t < t1; t++) {
        v16f s[1];
        v8bf p[2];
        const bool more = t + 2 < t1;
        if (more)
            wait_copies<3 * C>();
        else
            wait_copies<0>();
        st.template products<1, false, true>(vt, p, kt + (t & 1) * TILE, qf, s, lane);
        __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0): the tile is read before copies go over it
        stage_k(t + 2);
        st.template weigh<1>(s, p, a.c2, t * KW, t0 * KW, lim, t * KW + KW - 1 > low, lane);
        if (more)
            wait_copies<3 * C>();
        st.template products<1, true, false>(vt + (t & 1) * TILE, p, kt, qf, s, lane);
        __builtin_amdgcn_s_waitcnt(0xc07f);
        stage_v(t + 2);
    }
    // the waves' results: [column][D + 4] floats, output then maximum and sum
    constexpr int LD = D + 4;
    float *mine = reinterpret_cast<float *>(lds[wave]) + (lane & 31) * LD;
    const float l = st.l + other_half(st.l);
#pragma unroll
    for (int b = 0; b < D / 32; b++)
#pragma unroll
        for (int g = 0; g < 4; g++)
            *reinterpret_cast<float4 *>(mine + 32 * b + 8 * g + 4 * (lane >> 5)) =
                make_float4(st.o[b][4 * g], st.o[b][4 * g + 1], st.o[b][4 * g + 2], st.o[b][4 * g + 3]);
    if (lane < 32)
        *reinterpret_cast<float2 *>(mine + D) = make_float2(st.m, l);
    __syncthreads();
    constexpr int RUN = 8, PER = 64 * NW / (D / RUN);   // columns at a time, 8 elements a thread
    for (int cc = threadIdx.x / (D / RUN); cc < cols; cc += PER) {
        const int d = (threadIdx.x % (D / RUN)) * RUN;
        float m = kNoMax, sum = 0.0f, v[RUN];
#pragma unroll
        for (int w = 0; w < NW; w++)
            m = fmaxf(m, reinterpret_cast<const float *>(lds[w])[cc * LD + D]);
#pragma unroll
        for (int e = 0; e < RUN; e++)
            v[e] = 0.0f;
#pragma unroll
        for (int w = 0; w < NW; w++) {
            const float *p = reinterpret_cast<const float *>(lds[w]) + cc * LD;
            const float f = __builtin_amdgcn_exp2f(p[D] - m);
            sum = fmaf(f, p[D + 1], sum);
#pragma unroll
            for (int e = 0; e < RUN; e++)
                v[e] = fmaf(f, p[d + e], v[e]);
        }
        const int t = q.start + cc / group, hd = kh * group + cc % group;
        if (a.splits == 1) {
            const float f = reciprocal(sum);
            *reinterpret_cast<uint4 *>(a.o + (int64_t)t * a.ldo + hd * D + d) =
                make_uint4(to_bf16x2(v[0] * f, v[1] * f), to_bf16x2(v[2] * f, v[3] * f), to_bf16x2(v[4] * f, v[5] * f),
                           to_bf16x2(v[6] * f, v[7] * f));
            if (a.lse && d == 0)
                a.lse[(int64_t)hd * a.s.tokens_q + t] = log_sum(m, sum);
        } else {
            const int64_t p = part_row(a, split, hd, t);
            *reinterpret_cast<float4 *>(a.part + p * D + d) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(a.part + p * D + d + 4) = make_float4(v[4], v[5], v[6], v[7]);
            if (d == 0)
                a.stat[p] = make_float2(m, sum);
        }
    }
}

// The splits' shares of a row and head: o = sum 2^(m_s - m) o_s / sum 2^(m_s - m) l_s, eight shares' loads at a time
// (8 shares of 16 rows of 16 heads: 4.5 us; one share after the other 8.1).
template <int D>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnFwd a)
{
    constexpr int PER = 256 / (D / 4);   // rows and heads of a workgroup
    const int64_t n = (int64_t)blockIdx.x * PER + threadIdx.x / (D / 4), rows = (int64_t)a.s.max_q * a.s.hq;
    const int seq = (int)(n / rows), head = (int)(n % a.s.hq), i = (int)(n % rows / a.s.hq), d = (threadIdx.x % (D / 4)) * 4;
    if (seq >= a.s.seqs)
        return;
    const Rows q = q_rows(a.s, seq);
    if (i >= q.len)
        return;
    const int t = q.start + i;
    constexpr int AT = 8;
    float m = kNoMax, sum = 0.0f;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s0 = 0; s0 < a.splits; s0 += AT) {
        float2 st[AT];
        float4 o[AT];
#pragma unroll
        for (int u = 0; u < AT; u++) {
            const int64_t p = part_row(a, min(s0 + u, a.splits - 1), head, t);
            st[u] = a.stat[p];
            o[u] = *reinterpret_cast<const float4 *>(a.part + p * D + d);
        }
        float now = m;
#pragma unroll
        for (int u = 0; u < AT; u++)
            now = fmaxf(now, st[u].x);
        const float f = __builtin_amdgcn_exp2f(m - now);
        m = now;
        sum *= f;
        v = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
#pragma unroll
        for (int u = 0; u < AT; u++) {
            const float g = s0 + u < a.splits ? __builtin_amdgcn_exp2f(st[u].x - m) : 0.0f;
            sum = fmaf(g, st[u].y, sum);
            v = make_float4(fmaf(g, o[u].x, v.x), fmaf(g, o[u].y, v.y), fmaf(g, o[u].z, v.z), fmaf(g, o[u].w, v.w));
        }
    }
    const float f = reciprocal(sum);
    *reinterpret_cast<uint2 *>(a.o + (int64_t)t * a.ldo + head * D + d) =
        make_uint2(to_bf16x2(v.x * f, v.y * f), to_bf16x2(v.z * f, v.w * f));
    if (a.lse && d == 0)
        a.lse[(int64_t)head * a.s.tokens_q + t] = log_sum(m, sum);
}

// ---------------------------------------------------------------------------
// Gradient.  A first pass forms -L / c and -D of every row of a sequence and head, with which
// the two products S and dP start their accumulators: P is then 2^(c log2(e) S')
// and dS is P dP'.  Two kernels follow: keys' gradients (a workgroup owns keys and
// goes through the queries of the key head's group) and queries' gradients (it
// owns queries and goes through the keys).  S, P and dP are formed in both, seven
// products instead of five, so that no sum is added up in memory: results do not
// depend on the order workgroups run in.
// ---------------------------------------------------------------------------
// A wave takes 32 rows of one head.  D is sum P dP, and do o the same number with o's rounding to BF16 in it (half a
// step, 2^-8 of each term at most).  Where the weight is spread over many keys dq and dk do not notice (300 rows of
// normal q and k: 2.3e-3 off); where few keys share it, dP and D nearly cancel, and it is most of their error.  Rows that
// see at most FEW keys form the sum itself, from one tile of S and dP (lanes that walk over such a row's keys cost 8 us
// more at 2 x 4096 queries).  Longer rows keep it, also when their weight lies on a few keys: with q and k three and six
// times as large dq and dk are 4.4e-3 to 1.2e-2 off.  The sum itself would need every score once more here.  The rest is
// one read of o and do: 18 us for the 67 MB of 2 x 4096 queries, 16 heads of 128 (3.7 TB/s; a pass without the tile took
// 17).
constexpr int FEW = 32;
template <int D> __global__ __launch_bounds__(256) void attn_bwd_rows_kernel(AttnBwd a)
{
    using Lds = Tile<D>;
    constexpr int L = D / 8, R = 64 / L;   // lanes of a row, rows of a load
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    // sequences first, then heads, then rows; the grid's second dimension keeps the first one's threads below 2^32 where
    // sequences and query heads are many
    const unsigned at_grid = blockIdx.y * gridDim.x + blockIdx.x, seqs = (unsigned)a.s.seqs;
    const int heads = (int)gridDim.y, seq = uniform((int)(at_grid % seqs)), block = uniform((int)(at_grid / seqs));
    const int head = block % heads * 4 + wave, i0 = block / heads * 32;
    const Rows q = uniform(q_rows(a.s, seq)), k = uniform(k_rows(a.s, seq));
    if (head >= a.s.hq || i0 >= q.len)
        return;
    // Rows few .. most - 1 see 1 to FEW keys.
    const int shift = shift_of(q, k);
    const int few = a.s.causal ? max(0, -shift) : 0;
    const int most = k.len <= FEW ? q.len : a.s.causal ? min(q.len, FEW - shift) : 0;
    const int own = min(i0 + (lane & 31), q.len - 1);
    const int64_t at = (int64_t)head * a.s.tokens_q + q.start;
    const float lse = a.lse[at + own];
    const bool sees = lse != -INFINITY;   // rows that see nothing are masked everywhere
    if (i0 + lane == own)
        a.nl[at + own] = sees ? -lse / a.scale : 0.0f;
    if (k.len > 0 && i0 < most && i0 + 32 > few) {
        const int64_t t = q.start + own, j = k.start + min(lane & 31, k.len - 1);
        const int kv = head / (a.s.hq / a.s.hk);
        v16f s = splat(0.0f), dp = splat(0.0f);
        v8bf x[Lds::SLICES], y[Lds::SLICES];
        Lds::load(a.k + j * a.ldk + kv * D, lane, x);
        Lds::load(a.q + t * a.ldq + head * D, lane, y);
#pragma unroll
        for (int n = 0; n < Lds::SLICES; n++)
            s = mfma(x[n], y[n], s);
        Lds::load(a.v + j * a.ldv + kv * D, lane, x);
        Lds::load(a.dout + t * a.lddo + head * D, lane, y);
#pragma unroll
        for (int n = 0; n < Lds::SLICES; n++)
            dp = mfma(x[n], y[n], dp);
        const int lim = a.s.causal ? min(k.len - 1, own + shift) : k.len - 1;
        float sum = 0.0f;
#pragma unroll
        for (int e = 0; e < 16; e++) {
            const float p = __builtin_amdgcn_exp2f(fmaf(s[e], a.c2, -lse * kLog2e)) * dp[e];
            sum += acc_row(e, lane) > lim ? 0.0f : p;
        }
        sum += __shfl_xor(sum, 32, 64);
        if (i0 + lane == own && own >= few && own < most)
            a.nd[at + own] = sees ? -sum : 0.0f;
    }
    if (i0 >= few && i0 + 31 < most)
        return;
    const int64_t first = (int64_t)q.start * a.lddo + head * D + lane % L * 8;
    const int64_t first_o = (int64_t)q.start * a.ldo + head * D + lane % L * 8;
#pragma unroll
    for (int n = 0; n < 32; n += R) {
        const int i = i0 + n + lane / L, row = min(i, q.len - 1);
        float x[8], y[8], sum = 0.0f;
        Elem<uint16_t>::load8(a.o + first_o + row * a.ldo, x);
        Elem<uint16_t>::load8(a.dout + first + row * a.lddo, y);
#pragma unroll
        for (int e = 0; e < 8; e++)
            sum = fmaf(x[e], y[e], sum);
#pragma unroll
        for (int w = 1; w < L; w <<= 1)
            sum += __shfl_xor(sum, w, 64);
        if (lane % L == 0 && i < q.len && (i < few || i >= most))
            a.nd[at + i] = -sum;
    }
}

// Keys' and values' gradients: NW waves of 32 keys, HV times.  QT queries of one head at a time go through LDS; the
// HV waves of the same keys take every HV-th run of 32 of them, and their sums meet at the end.  Four waves of keys,
// twice, read a tile least often; where that makes few workgroups it is two waves, four times, or one, eight times
// (bwd_k_waves).  2 x 4096 causal queries, 16 heads of 128:
// 255 to 285 us for four products (275 GFLOP, 1.0 PFLOP/s), matrix cores busy 0.55 of the time, waits 0.31 of the waves'.
// Registers bound it: with K read from LDS and two waves a SIMD all 256 are in use, so that a third tile on its way or
// the exponentials beside the products' next run found no room (472 against 456 us in all; 302 against 255 alone).
template <int D, int NW, int HV>
__global__ __launch_bounds__(64 * NW * HV) void attn_bwd_k_kernel(AttnBwd a)
{
    constexpr int A1 = 4, A2 = 4, R = 32 * NW, QT = HV == 8 ? 256 : HV == 4 ? 128 : 8192 / D, TILE = Tile<D>::bytes(QT), STAGE = 2 * TILE + 2 * QT * 4, B = D / 32;
    static_assert(2 * STAGE >= HV / 2 * NW * 16 * B * 256, "half of one of the sums takes the tiles' place");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][STAGE], lds_k[Tile<D>::bytes(R)];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kw = wave % NW, part = wave / NW;
    const int units = a.s.seqs * a.s.hk, group = a.s.hq / a.s.hk;
    const int block = uniform((int)blockIdx.x / units), unit = (int)blockIdx.x - block * units;   // earlier keys, seen by more, first
    const int seq = uniform(unit / a.s.hk), kh = unit - seq * a.s.hk;
    const Rows q = uniform(q_rows(a.s, seq)), k = uniform(k_rows(a.s, seq));
    const int k0 = block * R;
    if (k0 >= k.len)
        return;
    const int shift = shift_of(q, k), tiles = (q.len + QT - 1) / QT;
    const int t0 = a.s.causal ? min(tiles, max(0, k0 - shift) / QT) : 0, steps = (tiles - t0) * group;

    const typename Tile<D>::template Stage<QT, HV * NW> copy_q(a.ldq, wave, lane), copy_d(a.lddo, wave, lane);
    int sh = kh * group, st = t0;   // the next tile to be copied: its head and its place
    auto stage = [&](int n) {
        const int last = q.len - 1 - st * QT;
        const int64_t row = (int64_t)q.start + st * QT;
        uint8_t *dst = lds[n & 1];
        copy_q(dst, a.q + row * a.ldq + sh * D, last, wave);
        copy_d(dst + TILE, a.dout + row * a.lddo + sh * D, last, wave);
        if (wave < QT / 64) {
            const uint32_t off = (uint32_t)min(64 * wave + lane, last) * 4;
            copy4(a.nl + (int64_t)sh * a.s.tokens_q + row, off, dst + 2 * TILE + 256 * wave);
            copy4(a.nd + (int64_t)sh * a.s.tokens_q + row, off, dst + 2 * TILE + QT * 4 + 256 * wave);
        }
        if (++st == tiles) {
            st = t0;
            sh++;
        }
    };
    if (steps > 0)
        stage(0);
    const int w0 = k0 + 32 * kw, j = w0 + (lane & 31), row = k.start + min(j, k.len - 1);
    // the values' operand stays in registers; the keys' is read from LDS again, which leaves registers for the reads
    // ahead
    constexpr int KW = R / Tile<D>::PIECE < HV * NW ? R / Tile<D>::PIECE : HV * NW;   // waves that copy K
    const typename Tile<D>::template Stage<R, KW> copy_k(a.ldk, wave, lane);
    if (wave < KW)
        copy_k(lds_k, a.k + (int64_t)(k.start + k0) * a.ldk + kh * D, k.len - 1 - k0, wave);
    v8bf vf[D / 16];
    Tile<D>::load(a.v + (int64_t)row * a.ldv + kh * D, lane, vf);
    pin(vf);
    const int from = a.s.causal ? j - shift : 0;              // the lane's first query
    const int wfirst = a.s.causal ? w0 - shift : 0, wlast = a.s.causal ? w0 + 31 - shift : 0;
    const int rb = Tile<D>::row_base(lane), cb = Tile<D>::col_base(lane);

    v16f dk[B], dv[B];
#pragma unroll
    for (int b = 0; b < B; b++)
        dk[b] = dv[b] = splat(0.0f);
    wait_copies<0>();   // where there are no steps, no copy outlives the workgroup
    int t = t0;
    for (int n = 0; n < steps; n++) {
        wait_copies<0>();
        __syncthreads();
        if (n + 1 < steps)
            stage(n + 1);
        const uint8_t *qt = lds[n & 1], *dt = qt + TILE;
        const float *nl = reinterpret_cast<const float *>(qt + 2 * TILE), *nd = nl + QT;
        const int i0 = t * QT;
        t = t + 1 == tiles ? t0 : t + 1;
#pragma unroll 1
        for (int u = part; u < QT / 32; u += HV) {
            const int i1 = i0 + 32 * u;
            if (i1 + 31 < wfirst || i1 >= q.len)
                continue;
            const uint8_t *qu = qt + u * Tile<D>::bytes(32), *du = dt + u * Tile<D>::bytes(32);
            v16f s, dp;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const float4 x = *reinterpret_cast<const float4 *>(nl + 32 * u + 8 * g + 4 * (lane >> 5));
                const float4 y = *reinterpret_cast<const float4 *>(nd + 32 * u + 8 * g + 4 * (lane >> 5));
                s[4 * g] = x.x; s[4 * g + 1] = x.y; s[4 * g + 2] = x.z; s[4 * g + 3] = x.w;
                dp[4 * g] = y.x; dp[4 * g + 1] = y.y; dp[4 * g + 2] = y.z; dp[4 * g + 3] = y.w;
            }
            struct Two {
                v8bf a, k;
            };
            constexpr int S = D / 16;
            Feed<2 * S, A1, Two> in;
            auto load_in = [&](auto I) {
                constexpr int n = decltype(I)::value;
                Two t;
                if constexpr (n % 2 == 0) {
                    t.a = Tile<D>::rows(qu + rb, 0, n / 2);
                    t.k = Tile<D>::rows(lds_k + kw * Tile<D>::bytes(32) + rb, 0, n / 2);
                } else {
                    t.a = t.k = Tile<D>::rows(du + rb, 0, n / 2);
                }
                return t;
            };
            in.first(load_in);
            in.run(load_in, [&](auto I, const Two &t) {
                constexpr int n = decltype(I)::value;
                if constexpr (n % 2 == 0)
                    s = mfma(t.a, t.k, s);
                else
                    dp = mfma(t.a, vf[n / 2], dp);
            });
            Feed<4 * B, A2> out;
            auto load_out = [&](auto I) {
                constexpr int n = decltype(I)::value;   // dv and dk in turn, block by block of both runs of 16 queries
                return Tile<D>::cols((n % 2 == 0 ? du : qu) + cb, 16 * (n / (2 * B)), n / 2 % B);
            };
            out.first(load_out);
            if (i1 < wlast || i1 + 32 > q.len) {
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const int i = i1 + acc_row(e, lane);
                    s[e] = i < from || i >= q.len ? -INFINITY : s[e];
                }
            }
            v8bf p[2], ds[2];
#pragma unroll
            for (int x = 0; x < 2; x++) {
#pragma unroll
                for (int e = 8 * x; e < 8 * x + 8; e++) {
                    s[e] = __builtin_amdgcn_exp2f(s[e] * a.c2);
                    dp[e] *= s[e];
                }
                p[x] = operand(s, x);
                ds[x] = operand(dp, x);
            }
            out.run(load_out, [&](auto I, const v8bf &x) {
                constexpr int n = decltype(I)::value, b = n / 2 % B, h = n / (2 * B);
                if constexpr (n % 2 == 0)
                    dv[b] = mfma(x, p[h], dv[b]);
                else
                    dk[b] = mfma(x, ds[h], dk[b]);
            });
        }
    }
    // dk is added up towards the first part, dv towards the last one
    float *const sums = reinterpret_cast<float *>(lds[0]) + lane;
    auto meet = [&](v16f (&v)[B], int place, int h) {
        float *x = sums + ((place < h ? place : place - h) * NW + kw) * 16 * B * 64;
        __syncthreads();
        if (place >= h && place < 2 * h) {
#pragma unroll
            for (int b = 0; b < B; b++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    x[(16 * b + e) * 64] = v[b][e];
        }
        __syncthreads();
        if (place < h) {
#pragma unroll
            for (int b = 0; b < B; b++)
#pragma unroll
                for (int e = 0; e < 16; e++)
                    v[b][e] += x[(16 * b + e) * 64];
        }
    };
#pragma unroll
    for (int h = HV / 2; h > 0; h /= 2) {
        meet(dk, part, h);
        meet(dv, HV - 1 - part, h);
    }
    if (j < k.len) {
        if (part == 0)
            store_row<D>(a.dk + (int64_t)row * a.lddk + kh * D, dk, a.scale, lane);
        if (part == HV - 1)
            store_row<D>(a.dv + (int64_t)row * a.lddv + kh * D, dv, 1.0f, lane);
    }
}

// Queries' gradients: NW waves of 32 rows (as in the forward), HV times, 64 keys at a time through LDS, 32 in a step.
// The two waves of the same rows take a half of every tile each, and their sums meet at the end.  2 x 4096 causal
// queries, 16 heads of 128: 185 to 210 us for three products (206 GFLOP, 1.05 PFLOP/s), matrix cores busy 0.57 of the
// time.  Two barriers a tile with a SIMD's waves in turns, which helps the forward, took 211 us against 189.
template <int D, int NW, int HV>
__global__ __launch_bounds__(64 * NW * HV) void attn_bwd_q_kernel(AttnBwd a)
{
    constexpr int R = 32 * NW, KT = 64, TILE = Tile<D>::bytes(KT), B = D / 32, S = D / 16;
    __shared__ __attribute__((aligned(16))) uint8_t lds[5][TILE];
    uint8_t(*const lds_k)[TILE] = lds, (*const lds_v)[TILE] = lds + 3;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int rw = wave % NW, part = wave / NW;
    const int units = a.s.seqs * a.s.hk, group = a.s.hq / a.s.hk;
    const int x = uniform((int)blockIdx.x / units), unit = (int)blockIdx.x - x * units;
    const int seq = uniform(unit / a.s.hk), kh = unit - seq * a.s.hk;
    const Rows q = uniform(q_rows(a.s, seq)), k = uniform(k_rows(a.s, seq));
    const int r0 = (a.q_blocks - 1 - x) * R;
    const int rows = q.len * group;   // (query, head) pairs, a query's heads side by side
    if (r0 >= rows)
        return;
    const int shift = shift_of(q, k), last = uniform((min(r0 + R, rows) - 1) / group);
    const int seen = a.s.causal ? max(0, min(k.len, last + 1 + shift)) : k.len;
    const int tiles = (seen + KT - 1) / KT;

    const uint16_t *kp = a.k + (int64_t)k.start * a.ldk + kh * D, *vp = a.v + (int64_t)k.start * a.ldv + kh * D;
    const typename Tile<D>::template Stage<KT, NW * HV> copy_k(a.ldk, wave, lane), copy_v(a.ldv, wave, lane);
    int at = 0;   // the K tile's place among three: the last tile's is read for one step into the next
    auto stage = [&](int t, int place) {
        const int last = k.len - 1 - t * KT;
        copy_k(lds_k[place], kp + (int64_t)t * KT * a.ldk, last, wave);
        copy_v(lds_v[t & 1], vp + (int64_t)t * KT * a.ldv, last, wave);
    };
    if (tiles > 0)
        stage(0, 0);
    const int w0 = r0 + 32 * rw, r = w0 + (lane & 31), rc = min(r, rows - 1);
    const int i = rc / group, head = kh * group + (rc - i * group), row = q.start + i;
    v8bf qf[S], df[S];
    Tile<D>::load(a.q + (int64_t)row * a.ldq + head * D, lane, qf);
    Tile<D>::load(a.dout + (int64_t)row * a.lddo + head * D, lane, df);
    pin(qf);
    pin(df);
    const float nl = a.nl[(int64_t)head * a.s.tokens_q + row] * a.c2, nd = a.nd[(int64_t)head * a.s.tokens_q + row];
    const int lim = a.s.causal ? min(k.len - 1, i + shift) : k.len - 1;
    // what the wave's first and last rows see
    const int low = a.s.causal ? min(k.len - 1, uniform(w0 / group) + shift) : k.len - 1;
    const int high = a.s.causal ? min(k.len - 1, uniform((w0 + 31) / group) + shift) : k.len - 1;
    const int rb = Tile<D>::row_base(lane), cb = Tile<D>::col_base(lane);

    v16f dq[B];
    v8bf ds[2];
#pragma unroll
    for (int b = 0; b < B; b++)
        dq[b] = splat(0.0f);
    ds[0] = ds[1] = __builtin_bit_cast(v8bf, v4u{0, 0, 0, 0});
    // a step: the last step's dS k (rows kc; zeros before the first one), and 32 keys' scores and dP
    auto add = [&](const uint8_t *kc) {
        feed<2 * B>([&](auto I) { return Tile<D>::cols(kc, 16 * (I / B), I % B); },
                    [&](auto I, const v8bf &f) { dq[I % B] = mfma(f, ds[I / B], dq[I % B]); });
    };
    auto step = [&](const uint8_t *kc, const uint8_t *kr, const uint8_t *vr, int j0) {
        v16f s = splat(0.0f), dp = splat(nd);
        feed<2 * B + 2 * S>(
            [&](auto I) {
                constexpr int n = decltype(I)::value;
                if constexpr (n < 2 * B)
                    return Tile<D>::cols(kc, 16 * (n / B), n % B);
                else if constexpr (n % 2 == 0)
                    return Tile<D>::rows(kr, 0, (n - 2 * B) / 2);
                else
                    return Tile<D>::rows(vr, 0, (n - 2 * B) / 2);
            },
            [&](auto I, const v8bf &f) {
                constexpr int n = decltype(I)::value;
                if constexpr (n < 2 * B)
                    dq[n % B] = mfma(f, ds[n / B], dq[n % B]);
                else if constexpr (n % 2 == 0)
                    s = mfma(f, qf[(n - 2 * B) / 2], s);
                else
                    dp = mfma(f, df[(n - 2 * B) / 2], dp);
            });
        if (j0 + 31 > low) {
#pragma unroll
            for (int e = 0; e < 16; e++)
                s[e] = j0 + acc_row(e, lane) > lim ? -INFINITY : s[e];
        }
#pragma unroll
        for (int e = 0; e < 16; e++)
            dp[e] *= __builtin_amdgcn_exp2f(fmaf(s[e], a.c2, nl));
        ds[0] = operand(dp, 0);
        ds[1] = operand(dp, 1);
    };
    constexpr int HALF = Tile<D>::bytes(32);
    const uint8_t *kc = lds_k[0] + cb;
    for (int t = 0; t < tiles; t++) {
        wait_copies<0>();
        __syncthreads();
        const int next = at == 2 ? 0 : at + 1;
        if (t + 1 < tiles)
            stage(t + 1, next);
#pragma unroll 1
        for (int u = part; u < 2; u += HV) {
            // one step past the wave's last visible key: it adds the step before and leaves zeros
            const int j0 = t * KT + 32 * u;
            const uint8_t *kt = lds_k[at] + u * HALF;
            if (j0 - 32 * HV <= high)
                step(kc, kt + rb, lds_v[t & 1] + u * HALF + rb, j0);
            kc = kt + cb;
        }
        at = next;
    }
    if (tiles > 0)
        add(kc);
    if constexpr (HV == 2) {
        constexpr int V = D / 2;   // a lane's values of dq
        static_assert(NW * V * 256 <= (int)sizeof(lds), "a half's sums take the tiles' place");
        float *x = reinterpret_cast<float *>(lds) + rw * V * 64 + lane;
        __syncthreads();
        if (part == 1) {
#pragma unroll
            for (int e = 0; e < V; e++)
                x[e * 64] = dq[e / 16][e % 16];
        }
        __syncthreads();
        if (part == 1)
            return;
#pragma unroll
        for (int e = 0; e < V; e++)
            dq[e / 16][e % 16] += x[e * 64];
    }
    if (r < rows)
        store_row<D>(a.dq + (int64_t)row * a.lddq + head * D, dq, a.scale, lane);
}

int64_t blocks_of(int64_t n, int64_t per) { return (n + per - 1) / per; }

// Rows of a key head: its queries of every query head.
int64_t rows_most(const AttnShape &s) { return (int64_t)s.max_q * (s.hq / s.hk); }

// Whether a key head's rows of every sequence fit one wave.  Then there is less to compute than to read.
bool few_rows(const AttnShape &s) { return rows_most(s) <= 32; }

// Workgroups of 128 rows of the forward: by the longest sequence, or by the rows there are.
int64_t fwd_groups(const AttnShape &s)
{
    const int64_t longest = (int64_t)s.seqs * s.hk * blocks_of(rows_most(s), 128);
    const int64_t rows = s.hk * (s.tokens_q * (s.hq / s.hk) / 128 + s.seqs);
    return longest < rows ? longest : rows;
}

// Shares of the key axis.  Few rows: as many as make 1024 workgroups (four a CU), of 512 keys or more (at least 256, 512
// and 1024 keys, 16 heads on 8 of 128: one sequence of 1000 keys 16, 18 and 18 us, of 4000 16, 16 and 25, eight of 4000
// 37.5, 36 and 36, one of 16000 23.5, 22 and 23.5; so a few sequences of up to 1023 keys are 2 us slower than they would
// be in shares).  Many rows: as many as make 256 workgroups of eight waves, one a CU, of 1024 keys or more (777 queries over
// 20000 keys, heads of 128: 135 us, unsplit 283, twice as many shares 157), but none where workgroups of 128 rows fill most
// CUs and the keys are not much longer than those workgroups' work (192 groups or more: 2048 x 2048 33 us, split 45; over
// 8192 keys 120 either way; 1500 x 17500 220, split 201), and none of up to 2048 keys (512 x 2048 32 us, split 35.5).
int splits_of(const AttnShape &s)
{
    if (s.seqs == 0 || s.max_q == 0)
        return 1;
    const int64_t units = (int64_t)s.seqs * s.hk;
    if (!few_rows(s) && (s.max_k <= 2048 || (s.max_k <= 8192 && fwd_groups(s) >= 192)))
        return 1;
    const int64_t groups = few_rows(s) ? units : units * blocks_of(rows_most(s), 256);
    int64_t want = groups ? (few_rows(s) ? 1024 : 256) / groups : 1;
    const int64_t most = s.max_k / (few_rows(s) ? 512 : 1024);
    want = want < most ? want : most;
    return (int)(want < 1 ? 1 : want > 64 ? 64 : want);
}

// Form of the forward's workgroups, NW x HV waves.  8 x 1 reads a tile for the most rows, and fills the card from some
// 640 workgroups of 128 rows on (2 x 3000 queries, heads of 128: 77 us, 4 x 1 78.6; 2 x 4096: 126, 141).  It is taken for
// keys in shares too: 777 queries over 20000 keys, 16 heads on 8: 135 us, 4 x 1 151, 4 x 2 158; 300 over 9000: 40, 43 and
// 51.  Where one block holds a key head's rows the others would be faster (100 queries over 9000 keys: 34, 30 and 27; 16
// times 5 over 9000, 16 heads on 2, 40 rows and six waves of copies of the last one: 41, 36 and 36).  Elsewhere below 640, smaller
// ones spread the rows over more CUs.  4 x 2 has a CU to itself and halves the way along the keys: for as many
// workgroups as CUs (1024 queries: 20 us, 4 x 1 23, 8 x 1 28), or twice as many where that way is long (4096: 73, 84 and
// 91).  4 x 1, two to a CU, for the rest (packed lengths 1 to 1500, heads of 64: 24.9 us, 4 x 2 30, 8 x 1 28.8).
enum Form { EIGHT, FOUR, FOUR_TWICE };
Form form_of(const AttnShape &s)
{
    const int64_t groups = fwd_groups(s);
    if (splits_of(s) > 1 || groups > 640)
        return EIGHT;
    return groups <= 256 || (groups <= 512 && s.max_k >= 2048) ? FOUR_TWICE : FOUR;
}

// Whether the queries' gradients take 128 rows a workgroup, every row's keys on two waves, instead of 256 (one CU each
// either way): where that leaves no more than one and a half workgroups a CU, or two with many keys.  The whole gradient,
// heads of 128: 1024 queries 83 -> 69 us, 4096 345 -> 306, 3 x 1024 94 -> 86; but 3 x 1500 155 -> 157, and packed
// lengths of 1 to 1500 (472 workgroups, heads of 64) 104 -> 111.
bool bwd_q_twice(const AttnShape &s)
{
    const int64_t groups = fwd_groups(s);
    return groups <= 384 || (groups <= 512 && s.max_k >= 2048);
}

// Waves of 32 keys of the keys' gradients: four, or two where four would make fewer workgroups (one a CU) than go over
// the CUs twice, by the longest sequence or by the rows there are.  The whole gradient with two and with four, heads of
// 128: 1024 queries 69 and 89 us, 4096 252 and 305, 2 x 4096 (512 workgroups) 481 and 456, 8 x 1024 189 and 169.
// One, eight times, where heads of 64 leave LDS for 256 queries a tile and it makes no more than two workgroups a CU: 12
// heads on 4 of 64, one and two: 1024 queries 43 and 52 us, 4096 133 and 157, 8192 445 and 409 (16 on 8: 3 x 1024 62
// and 53).
int bwd_k_waves(const AttnShape &s)
{
    const int64_t longest = (int64_t)s.seqs * s.hk * blocks_of(s.max_k, 128), rows = s.hk * (s.tokens_k / 128 + s.seqs);
    const int64_t groups = longest < rows ? longest : rows;
    return groups >= 512 ? 4 : s.dim == 64 && groups <= 128 && longest < 1 << 20 ? 1 : 2;
}

// Workgroups of the gradient's first pass for four heads, of 32 rows each.
int64_t bwd_row_groups(const AttnShape &s) { return s.seqs * blocks_of(s.max_q, 32); }

size_t pad256(size_t n) { return (n + 255) / 256 * 256; }

size_t part_bytes(const AttnShape &s, int splits) { return pad256((size_t)splits * s.hq * s.tokens_q * s.dim * 4); }

template <int D> hipError_t fwd(AttnFwd a, hipStream_t st)
{
    const int64_t units = (int64_t)a.s.seqs * a.s.hk;
    if (few_rows(a.s)) {
        hipLaunchKernelGGL((attn_rows_kernel<D>), dim3((unsigned)(units * a.splits)), dim3(64 * ROW_WAVES), 0, st, a);
    } else {
        const Form form = form_of(a.s);
        auto *kernel = form == EIGHT ? attn_fwd_kernel<D, 8, 1> : form == FOUR ? attn_fwd_kernel<D, 4, 1> : attn_fwd_kernel<D, 4, 2>;
        a.blocks = (int)blocks_of(rows_most(a.s), form == EIGHT ? 256 : 128);
        hipLaunchKernelGGL(kernel, dim3((unsigned)(units * a.splits * a.blocks)), dim3(form == FOUR ? 256 : 512), 0, st, a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.splits == 1)
        return e;
    const int64_t rows = (int64_t)a.s.seqs * a.s.max_q * a.s.hq;
    hipLaunchKernelGGL((attn_join_kernel<D>), dim3((unsigned)blocks_of(rows, 256 / (D / 4))), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int D> hipError_t bwd(AttnBwd b, hipStream_t st)
{
    const int64_t units = (int64_t)b.s.seqs * b.s.hk;
    hipError_t e = hipSuccess;
    if (b.s.max_q > 0) {
        hipLaunchKernelGGL((attn_bwd_rows_kernel<D>), dim3((unsigned)bwd_row_groups(b.s), (unsigned)blocks_of(b.s.hq, 4)),
                           dim3(256), 0, st, b);
        e = hipGetLastError();
    }
    if (e == hipSuccess && b.s.max_k > 0) {
        const int waves = bwd_k_waves(b.s);
        auto *kernel = waves == 4 ? attn_bwd_k_kernel<D, 4, 2> : attn_bwd_k_kernel<D, 2, 4>;
        if constexpr (D == 64)
            kernel = waves == 1 ? attn_bwd_k_kernel<D, 1, 8> : kernel;
        hipLaunchKernelGGL(kernel,
                           dim3((unsigned)(units * blocks_of(b.s.max_k, 32 * waves))), dim3(512), 0, st, b);
        e = hipGetLastError();
    }
    if (e == hipSuccess && b.s.max_q > 0) {
        const bool twice = bwd_q_twice(b.s);
        b.q_blocks = (int)blocks_of(rows_most(b.s), twice ? 128 : 256);
        hipLaunchKernelGGL((twice ? attn_bwd_q_kernel<D, 4, 2> : attn_bwd_q_kernel<D, 8, 1>),
                           dim3((unsigned)(units * b.q_blocks)), dim3(512), 0, st, b);
        e = hipGetLastError();
    }
    return e;
}

} // namespace

// Whether every launch stays below 2^32 threads along the grid's first dimension.
bool attn_fits(const AttnShape &s, bool backward)
{
    const double units = (double)s.seqs * s.hk, most = 4294967295.0;
    if (rows_most(s) > 1 << 30 || units > most)
        return false;
    auto threads = [&](int64_t blocks, int each) { return units * (double)blocks * each; };
    if (backward)
        return (double)bwd_row_groups(s) * 256 <= most && threads(blocks_of(s.max_k, 32 * bwd_k_waves(s)), 512) <= most &&
               threads(blocks_of(rows_most(s), bwd_q_twice(s) ? 128 : 256), 512) <= most;
    const int splits = splits_of(s);
    const double join = splits == 1 ? 0.0 : (double)s.seqs * s.hq * s.max_q * (s.dim / 4) + 256;
    if (few_rows(s))
        return threads(splits, 64 * ROW_WAVES) <= most && join <= most;
    const Form form = form_of(s);
    return threads(blocks_of(rows_most(s), form == EIGHT ? 256 : 128) * splits, form == FOUR ? 256 : 512) <= most && join <= most;
}

size_t attn_workspace_bytes(const AttnShape &s)
{
    const int splits = splits_of(s);
    return splits == 1 ? 0 : part_bytes(s, splits) + pad256((size_t)splits * s.hq * s.tokens_q * sizeof(float2));
}

hipError_t launch_attn(AttnFwd a, void *workspace, hipStream_t st)
{
    a.c2 = a.scale * kLog2e;
    a.splits = splits_of(a.s);
    a.part = (float *)workspace;
    a.stat = a.splits == 1 ? nullptr : (float2 *)((char *)workspace + part_bytes(a.s, a.splits));
    return a.s.dim == 64 ? fwd<64>(a, st) : fwd<128>(a, st);
}

size_t attn_bwd_workspace_bytes(const AttnShape &s) { return 2 * pad256((size_t)s.hq * s.tokens_q * 4); }

hipError_t launch_attn_bwd(AttnBwd b, void *workspace, hipStream_t st)
{
    b.c2 = b.scale * kLog2e;
    b.nl = (float *)workspace;
    b.nd = (float *)((char *)workspace + attn_bwd_workspace_bytes(b.s) / 2);
    return b.s.dim == 64 ? bwd<64>(b, st) : bwd<128>(b, st);
}

} // namespace puro
