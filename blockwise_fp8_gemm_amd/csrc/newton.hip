// Newton-Schulz orthogonalisation of weight gradients on the gfx950 matrix
// cores: the update direction of the Muon-type optimiser that the Puro-2B
// pages name for the recipe's matrix parameters.
//
// With M <= N (a tall matrix is handled as its transpose), X0 = G / (|G|_F +
// eps) and per step
//   A = X X^T,   B = b A + c A A,   X <- a X + B X
// which maps every singular value s of X to a s + b s^3 + c s^5 and leaves the
// singular vectors as they are.
//
// Number formats.  The products run on the FP16 matrix cores (BF16's rate,
// three more significand bits).  X is kept as the sum of two FP16 numbers, hi +
// lo: the products read hi, the term a X reads both.  Below 2^-2 lo lies in FP16's
// subnormals, so an entry is held to 2^-22 of itself or to 2^-25, whichever is
// more: 22 bits for scaled entries near one, as they are after the steps, 19 to 20
// for a first step's at 2048 x 2048 (near 2^-5.5).  The diagonal
// of B is kept apart in FP32 and joins a in that term, X <- (a + d_i) X +
// (B - d) hi, so that the part of the step that is largest for well
// conditioned rows carries no FP16 rounding at all.  X is held times a power
// of two near sqrt(N) and A and B times 2^10, which keeps entries clear of
// FP16's subnormals; with the singular values at most 2 and |b l + c l^2| at
// most 32 (checked on the host) nothing overflows.  Measured against 64 bits
// after five steps, on gradient-like, power-law, row-scaled and low-rank spectra
// from 700 x 300 to 6144 x 2048: 0.06e-3 to 1.4e-3 relative (Frobenius), the BF16
// rounding of the result itself being 1.66e-3; with BF16 operands 0.5e-2 to
// 1.6e-2 (simulated), with FP32 products far below the rounding, at a fraction of
// the rate: there is no such form.
//
// A and B are symmetric: only the tiles on and above the diagonal are formed,
// and each is stored twice.  In B X, X is contiguous along N and not along K: its
// fragments come through the LDS's transposing reads, which saves keeping
// (and writing, every step) a transposed copy of X.
#include "common.h"
#include "kernels.h"
#include "stores.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

namespace puro {

namespace {

typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));

constexpr float kScaleA = 1024.0f;   // A and B are held times this
constexpr int kNormBlocks = 256;     // partial sums of |G|^2 per matrix

// One 128-byte line: a kernel fetches its matrix's in one go.
struct alignas(128) NsItem {
    const void *g;
    void *o;
    int64_t ldg, ldo;
    int M, N;      // M <= N after the transpose of a tall matrix
    int Mp, Np;    // padded to whole tiles; the padding holds zeros
    int tall;
    float s;       // X is held times s
    uint16_t *xh[2], *xl;   // [Mp][Np]; hi is read from the first and written to the second
    uint16_t *a, *b;        // [Mp][Mp]
    float *d;               // [Mp] diagonal of B
    double *part;           // [kNormBlocks]
};

static_assert(sizeof(NsItem) == 128, "one line");

struct NsGroup {
    int first[kNsGroupMax + 1];   // workgroups of item i: [first[i], first[i+1]); past the last item, INT_MAX
    int count;
    int gbf16;
    int last;                     // the step whose result is the output
    float a, b, c, eps;
    NsItem it[kNsGroupMax];
};

typedef __attribute__((address_space(4))) const NsGroup *KernargNs;

__device__ __forceinline__ KernargNs kernarg()
{
    return (KernargNs)__builtin_amdgcn_kernarg_segment_ptr();
}

// The item that holds workgroup b.  All of `first` is read at once and compared
// without a loop: the arguments come from memory, and loads that wait for each
// other are a good part of a small launch's time.
__device__ __forceinline__ int find_item(KernargNs g, int b, int &begin, int &end)
{
    int i = 0;
    begin = 0;
    end = g->first[1];
#pragma unroll
    for (int k = 1; k < kNsGroupMax; k++) {
        const bool past = b >= g->first[k];
        i += past;
        begin = past ? g->first[k] : begin;
        end = past ? g->first[k + 1] : end;
    }
    return __builtin_amdgcn_readfirstlane(i);
}

// An FP32 value as it stands: keeps the compiler from folding the operation
// that made it into the conversion to FP16 (v_fma_mixlo rounds once where an
// FP32 result is rounded twice), which it does in one place and not in the
// next, so that the two stored copies of an element could differ.
__device__ __forceinline__ float as_f32(float f)
{
    asm("" : "+v"(f));
    return f;
}

// Values of the arguments, fetched together and kept: left alone the compiler
// loads each where it is used, and waits for it there (three small matrices 92
// against 88 us, B X of a layer's gradients 213 against 211).
template <typename T> __device__ __forceinline__ void keep(T *&p)
{
    uint64_t v = (uint64_t)p;
    asm volatile("" : "+s"(v));
    p = (T *)(__attribute__((address_space(1))) T *)v;
}
__device__ __forceinline__ void keep(int &v) { asm volatile("" : "+s"(v)); }
__device__ __forceinline__ void keep(int64_t &v) { asm volatile("" : "+s"(v)); }
__device__ __forceinline__ void keep(float &v) { asm volatile("" : "+s"(v)); }
template <typename... T> __device__ __forceinline__ void keep_all(T &...v) { (keep(v), ...); }

// ---------------------------------------------------------------------------
// |G|_F^2 in 64 bits: kNormBlocks partial sums per matrix.  A wave takes a row
// at a time, 16 bytes a lane.
// ---------------------------------------------------------------------------
template <typename T> __device__ __forceinline__ double row_squares(const T *row, int cols, int lane)
{
    constexpr int V = 16 / sizeof(T);
    double s0 = 0.0, s1 = 0.0;
#pragma unroll 4
    for (int c = lane * V; c < cols; c += 64 * V) {
        float v[8];
        if (c + V <= cols) {
            if constexpr (V == 8) {
                Elem<T>::load8(row + c, v);
            } else {
                const float4 f = *reinterpret_cast<const float4 *>(row + c);
                v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
            }
        } else {
#pragma unroll
            for (int k = 0; k < V; k++)
                v[k] = c + k < cols ? Elem<T>::load(row + c + k) : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < V; k += 2) {
            s0 = fma((double)v[k], (double)v[k], s0);
            s1 = fma((double)v[k + 1], (double)v[k + 1], s1);
        }
    }
    return s0 + s1;
}

__global__ __launch_bounds__(256) void ns_norm_kernel(NsGroup args)
{
    (void)args;
    const KernargNs g = kernarg();
    const int item = blockIdx.y, t = threadIdx.x;
    const int tall = g->it[item].tall;
    const int rows = tall ? g->it[item].N : g->it[item].M, cols = tall ? g->it[item].M : g->it[item].N;
    const int64_t ld = g->it[item].ldg;
    const void *src = g->it[item].g;
    __shared__ double red[256];
    double sum = 0.0;
    for (int r = blockIdx.x * 4 + (t >> 6); r < rows; r += kNormBlocks * 4)
        sum += g->gbf16 ? row_squares((const uint16_t *)src + r * ld, cols, t & 63)
                        : row_squares((const float *)src + r * ld, cols, t & 63);
    red[t] = sum;
    __syncthreads();
    for (int w = 128; w > 0; w >>= 1) {
        if (t < w)
            red[t] += red[t + w];
        __syncthreads();
    }
    if (t == 0)
        g->it[item].part[blockIdx.x] = red[0];
}

// ---------------------------------------------------------------------------
// X0: hi and lo of a 64 x 64 tile, zeros in the padding.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void ns_init_kernel(NsGroup args)
{
    (void)args;
    const KernargNs g = kernarg();
    int begin, end;
    const int i = find_item(g, blockIdx.x, begin, end), t = threadIdx.x;
    const int local = blockIdx.x - begin;
    const int M = g->it[i].M, N = g->it[i].N, Np = g->it[i].Np, tall = g->it[i].tall;
    const int rows = tall ? N : M, cols = tall ? M : N;
    const int64_t ld = g->it[i].ldg;
    const int m0 = local / (Np / 64) * 64, n0 = local % (Np / 64) * 64;
    const int r0 = tall ? n0 : m0, c0 = tall ? m0 : n0;
    __shared__ double red[4];
    __shared__ float x[64][64 + 1];   // as the source lies
    // thread t takes 16 elements of row t / 4, eight at a time; a tall source goes through LDS
    const int q = t >> 2, r = r0 + q;
    double sum = g->it[i].part[t];
    static_assert(kNormBlocks == 256, "a partial sum per thread");
    float v[2][8];
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const int c = c0 + 16 * (t & 3) + 8 * h;
        if (r < rows && c + 8 <= cols) {
            if (g->gbf16)
                Elem<uint16_t>::load8((const uint16_t *)g->it[i].g + r * ld + c, v[h]);
            else
                Elem<float>::load8((const float *)g->it[i].g + r * ld + c, v[h]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++) {
                v[h][k] = 0.0f;
                if (r < rows && c + k < cols)
                    v[h][k] = g->gbf16 ? Elem<uint16_t>::load((const uint16_t *)g->it[i].g + r * ld + c + k)
                                       : ((const float *)g->it[i].g)[r * ld + c + k];
            }
        }
    }
    // the norm, while the elements are on their way
#pragma unroll
    for (int k = 1; k < 64; k <<= 1)
        sum += __shfl_xor(sum, k, 64);
    if ((t & 63) == 0)
        red[t >> 6] = sum;
    if (tall) {
#pragma unroll
        for (int h = 0; h < 2; h++)
#pragma unroll
            for (int k = 0; k < 8; k++)
                x[q][16 * (t & 3) + 8 * h + k] = v[h][k];
    }
    __syncthreads();
    // s / (|G| + eps) lies between 2^-142 and 2^156, past what one FP32 number holds at both ends:
    // two factors, a power of two (exact: it brings no element past s, and what it takes below FP32's
    // normal range is far below the last bit of lo) and a number of that size's square root
    int e;
    const double m = frexp((double)g->it[i].s / (sqrt(red[0] + red[1] + red[2] + red[3]) + (double)g->eps), &e);
    const float shift = ldexpf(1.0f, e / 2), scale = ldexpf((float)m, e - e / 2);
#pragma unroll
    for (int h = 0; h < 2; h++) {
        if (tall) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                v[h][k] = x[16 * (t & 3) + 8 * h + k][q];
        }
        const int64_t at = (int64_t)(m0 + q) * Np + n0 + 16 * (t & 3) + 8 * h;
        v8h hi, lo;
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float y = as_f32(v[h][k] * shift * scale);
            hi[k] = (_Float16)y;
            lo[k] = (_Float16)as_f32(y - (float)hi[k]);
        }
        *reinterpret_cast<v8h *>(g->it[i].xh[0] + at) = hi;
        *reinterpret_cast<v8h *>(g->it[i].xl + at) = lo;
    }
}

// ---------------------------------------------------------------------------
// Products.  A workgroup computes a TM x TN tile of P Q^T (P [..][K], Q [..][K],
// rows contiguous along K) with WM x WN waves of IT x JT matrix-core tiles of
// 16 x 16.  Blocks of 64 K (128 bytes a row) go from global memory straight to
// LDS, double-buffered, with a 16-byte XOR swizzle that keeps the 16-byte
// fragment reads free of bank conflicts.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t lds_addr(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// 16 bytes per lane from base + off (base wave-uniform) to the wave's LDS base
// + 16 lane.  Inline assembly rather than the builtin: with the builtin's copy
// in flight the compiler waits for every LDS read with lgkmcnt(0).  The copies
// count in vmcnt, which the K loop waits on before its barrier.  M0 is set in
// the same statement, one wait state ahead as LDS copies want it, and nothing
// else here reads it.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void copy16(const uint8_t *base, uint32_t off, uint8_t *lds_wave_base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(lds_addr(lds_wave_base)) : "memory", "m0");
}
#pragma clang diagnostic pop

// 16-byte segment s of row r sits at s ^ swz(r).
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Chunk `it` of this wave's share of ROWS rows: g is the block's first row at its first K.
template <int ROWS, int NW>
__device__ __forceinline__ void stage_rows(uint8_t *t, const uint8_t *g, uint32_t ld, int it, int wave, int lane)
{
    static_assert((ROWS / 8) % NW == 0, "whole 1 KB chunks per wave");
    const int c = wave + NW * it;   // rows 8c .. 8c+7, lane's row 8c + lane / 8
    const int seg = (lane & 7) ^ (((lane >> 3) & 7) ^ (c & 1));
    copy16(g, (uint32_t)(8 * c + (lane >> 3)) * ld + (uint32_t)(seg * 16), t + c * 1024);
}

// Rows row_base + lane % 16, K values 16 (lane / 16) .. +15 of a 64-wide block
// (the same K slots in both operands, so any order of K serves).
struct Frag {
    v8h k[2];
};
__device__ __forceinline__ Frag frag(const uint8_t *t, int row_base, int lane)
{
    const int row = row_base + (lane & 15);
    const int g = lane >> 4, f = swz(row);
    Frag r;
    r.k[0] = __builtin_bit_cast(v8h, *reinterpret_cast<const v4i *>(t + (row * 128 + (((2 * g) ^ f) << 4))));
    r.k[1] = __builtin_bit_cast(v8h, *reinterpret_cast<const v4i *>(t + (row * 128 + (((2 * g + 1) ^ f) << 4))));
    return r;
}

// The same for an operand that is contiguous along its rows' dimension: 64 rows
// of K, W elements each.  A transposing read takes 4 K rows x 16 elements per 16
// lanes; the swizzle puts the 16 pieces of 32 bytes that a wave reads at once
// (4 rows of 4 lane groups) on different banks.
__device__ __forceinline__ int swz_k(int k) { return ((k & 3) << 1) | (((k >> 4) & 1) << 3) | (((k >> 5) & 1) << 4); }

template <int W> __device__ __forceinline__ int swz_kw(int k) { return swz_k(k) & (W / 8 - 1); }

template <int W, int NW>
__device__ __forceinline__ void stage_k(uint8_t *t, const uint8_t *g, uint32_t ld, int it, int wave, int lane)
{
    constexpr int SEGS = W / 8, RPC = 64 / SEGS;   // 16-byte segments per row, rows per 1 KB chunk
    static_assert((64 / RPC) % NW == 0, "whole 1 KB chunks per wave");
    const int c = wave + NW * it, row = RPC * c + lane / SEGS;
    const int seg = (lane % SEGS) ^ swz_kw<W>(row);
    copy16(g, (uint32_t)row * ld + (uint32_t)(seg * 16), t + c * 1024);
}

template <int W> __device__ __forceinline__ Frag frag_k(const uint8_t *t, int col_base, int lane)
{
    typedef __attribute__((address_space(3))) v4s lds_v4s;
    const int i = lane & 15, g = lane >> 4;
    Frag r;
#pragma unroll
    for (int kk = 0; kk < 2; kk++) {
        v4s q[2];
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const int k = 16 * g + 8 * kk + 4 * h + (i >> 2), col = col_base * 2 + 8 * (i & 3);
            q[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lds_v4s *)(t + (k * (2 * W) + (((col >> 4) ^ swz_kw<W>(k)) << 4) + (col & 8))));
        }
        r.k[kk] = __builtin_bit_cast(v8h, __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
    return r;
}

// WM x WN waves of IT x JT tiles of 16 x 16; S stages of 64 K in LDS.
template <int WM_, int WN_, int IT_, int JT_, int S_> struct NsCfg {
    static constexpr int WM = WM_, WN = WN_, IT = IT_, JT = JT_, S = S_;
    static constexpr int NW = WM * WN, THREADS = 64 * NW;
    static constexpr int TM = WM * IT * 16, TN = WN * JT * 16;
    static constexpr int STAGE = (TM + TN) * 128, LOADS = (TM + TN) / 8 / NW;
    static constexpr int SPAN = IT * 16;           // elements of a result row per wave
    static constexpr int TURN = SPAN * 64;         // bytes of each of a wave's two epilogue buffers
    // the low halves go past the caches where the many tiles of the large form leave them no
    // use there (B X of a layer's seven gradients 221 -> 216 us); one 2048 x 2048 matrix on
    // 128 x 128 tiles keeps them (26.9, and 27.6 past the caches)
    static constexpr bool STREAM = TM * TN == 256 * 256;
    static_assert(S * STAGE >= NW * 2 * TURN, "the epilogue's buffers take the stages' place");
};
// The large tile reads least from LDS per product; the smaller ones fill the GPU
// where there are few tiles or some are deep, and have LDS left for a third and
// fourth stage.  Eight waves (two per SIMD) on the three large ones: with four the
// two smaller of them took a fifth to a third longer; four waves of 128 x 128 on the
// largest run their K loop at the matrix cores' rate (0.94 us a block instead of
// 1.00), but alone on their SIMDs lose more in the epilogue (A A of a layer's
// gradients 59 us instead of 54).
typedef NsCfg<2, 4, 8, 4, 2> NsL;   // 256 x 256
typedef NsCfg<4, 2, 4, 4, 3> NsM;   // 256 x 128
typedef NsCfg<2, 4, 4, 2, 4> NsQ;   // 128 x 128
typedef NsCfg<2, 2, 2, 2, 4> NsE;   // 64 x 64

enum { NS_GRAM = 0, NS_POLY = 1, NS_UPDATE = 2 };

// Workgroups are dispatched round-robin over the 8 XCDs.  Of the workgroups
// [first, end) of one matrix, those on XCD x take a contiguous run of its tiles,
// so that the tiles resident together on one XCD read the same operand panels
// through its L2, and every XCD has its share of every matrix.
__device__ __forceinline__ int xcd_local(int b, int first, int end)
{
    const int x = b & 7;
    // workgroups of [0, n) on the XCDs before x, and on x itself
    auto before = [x](int n) { return (n >> 3) * x + min(n & 7, x); };
    auto on = [x](int n) { return (n - x + 7) >> 3; };
    return before(end) - before(first) + on(b) - on(first);
}

// Eight 16-bit values to row[c0 ..], those before cols.
__device__ __forceinline__ void store_run(uint16_t *row, int c0, int cols, const uint32_t w[4])
{
    if (c0 + 8 <= cols) {
        store_nt(row + c0, w[0], w[1], w[2], w[3]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; k++)
        if (c0 + k < cols)
            row[c0 + k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
}

template <int N> __device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// f(0) .. f(N - 1) with constant arguments.
template <int N, class F> __device__ __forceinline__ void each(F f)
{
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

template <class Cfg, int MODE>
__global__ __launch_bounds__(Cfg::THREADS) void ns_product_kernel(NsGroup args)
{
    (void)args;
    constexpr int NW = Cfg::NW, TM = Cfg::TM, TN = Cfg::TN, IT = Cfg::IT, JT = Cfg::JT, S = Cfg::S;
    __shared__ __attribute__((aligned(16))) uint8_t lds[S * Cfg::STAGE];
    const KernargNs g = kernarg();
    int begin, end;
    const int item = find_item(g, blockIdx.x, begin, end);
    const int local = xcd_local(blockIdx.x, begin, end);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
    int Mp = g->it[item].Mp, Np = g->it[item].Np, M = g->it[item].M, N = g->it[item].N, tall = g->it[item].tall;
    int last = g->last;
    int64_t ldo = g->it[item].ldo;
    float s = g->it[item].s, ga = g->a, gb = g->b, gc = g->c;
    uint16_t *xin = g->it[item].xh[0], *xout = g->it[item].xh[1], *xlow = g->it[item].xl, *ma = g->it[item].a,
             *mb = g->it[item].b, *result = (uint16_t *)g->it[item].o;
    float *diag = g->it[item].d;
    if constexpr (MODE == NS_GRAM)
        keep_all(Mp, Np, s, xin, ma);
    else if constexpr (MODE == NS_POLY)
        keep_all(Mp, gb, gc, ma, mb, diag);
    else
        keep_all(Mp, Np, M, N, tall, last, ldo, s, ga, xin, xout, xlow, mb, result, diag);

    // operands and the tile's place: P along the tile's rows, Q along its columns
    const uint8_t *P, *Q;
    int K, tr, tc;
    if constexpr (MODE == NS_UPDATE) {
        // the result's transpose: rows are X's columns (X [Mp][Np]), columns X's rows (B [Mp][Mp])
        P = (const uint8_t *)xin;
        Q = (const uint8_t *)mb;
        K = Mp;
        // strips of four tile columns, so that an XCD's run of tiles is nearly square and reads few
        // panels of both (a layer's gradients: 656 MB fetched instead of 801, 210 us instead of 212)
        const int R = Np / TM, C = Mp / TN, strip = local / (4 * R), w = min(4, C - 4 * strip);
        tr = (local - 4 * R * strip) / w;
        tc = 4 * strip + (local - 4 * R * strip) % w;
    } else {
        P = Q = (const uint8_t *)(MODE == NS_GRAM ? xin : ma);
        K = MODE == NS_GRAM ? Np : Mp;
        // tiles that reach the diagonal or lie above it, row by row of tiles
        tr = 0;
        tc = local;
        for (int left = Mp / TN; tc >= left; left -= TM / TN, tr++)
            tc -= left;
        tc += tr * (TM / TN);
    }
    const int64_t ldp = (int64_t)(MODE == NS_UPDATE ? Np : K) * 2, ldq = (int64_t)K * 2;
    const int m0 = tr * TM, n0 = tc * TN, KB = K / 64;

    v4f acc[IT][JT];
#pragma unroll
    for (int i = 0; i < IT; i++)
#pragma unroll
        for (int j = 0; j < JT; j++)
            acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    // Copy n of this wave's share of block kb into its stage; past the end the last
    // block again (never read), so that the number of copies in flight is the same
    // at every block.
    constexpr int PLOADS = TM / 8 / NW;
    const uint8_t *P0 = P + (MODE == NS_UPDATE ? (int64_t)m0 * 2 : m0 * ldp), *Q0 = Q + n0 * ldq;
    const int64_t pstep = MODE == NS_UPDATE ? 64 * ldp : 128;
    auto stage = [&](int kb, int n) {
        uint8_t *L = lds + kb % S * Cfg::STAGE;
        const int k = min(kb, KB - 1);
        if (n >= PLOADS)
            stage_rows<TN, NW>(L + TM * 128, Q0 + k * 128, (uint32_t)ldq, n - PLOADS, wave, lane);
        else if constexpr (MODE == NS_UPDATE)
            stage_k<TM, NW>(L, P0 + k * pstep, (uint32_t)ldp, n, wave, lane);
        else
            stage_rows<TM, NW>(L, P0 + k * pstep, (uint32_t)ldp, n, wave, lane);
    };
    auto read_p = [&](int kb, int i) {
        const uint8_t *L = lds + kb % S * Cfg::STAGE;
        if constexpr (MODE == NS_UPDATE)
            return frag_k<TM>(L, (wm * IT + i) * 16, lane);
        else
            return frag(L, (wm * IT + i) * 16, lane);
    };
    auto read_q = [&](int kb, int j) {
        return frag(lds + kb % S * Cfg::STAGE + TM * 128, (wn * JT + j) * 16, lane);
    };

    // The K loop.  All of a block's fragments are in registers two row blocks
    // before its end; there the waves meet, block kb + S is copied over the
    // stage just read, and the next block's first fragments are read.  Every
    // copy and read has its place between two products, held there by the
    // scheduling barriers: in front of a row block's products, where the compiler
    // gathers them, they leave the matrix cores idle (X X^T of a layer's
    // gradients 122 against 114 us, B X 208 against 200, one 2048 x 2048 20.5
    // and 27.7 against 18.8 and 25.6).
    Frag q[2][JT], p[2];
#pragma unroll
    for (int k = 0; k < S; k++)
#pragma unroll
        for (int n = 0; n < Cfg::LOADS; n++)
            stage(k, n);
    wait_copies<(S - 1) * Cfg::LOADS>();
    __syncthreads();
#pragma unroll
    for (int j = 0; j < JT; j++)
        q[0][j] = read_q(0, j);
    p[0] = read_p(0, 0);
    p[1] = read_p(0, 1);
    auto block = [&](int kb, Frag (&cur)[JT], Frag (&nxt)[JT]) {
        Frag np[2];
        each<IT>([&](auto I) {
            constexpr int i = decltype(I)::value, h = i - (IT - 2), N = 2 * JT;
            const Frag a = p[i & 1];
            if constexpr (h == 0) {
                wait_copies<(S - 2) * Cfg::LOADS>();
                __syncthreads();
            }
            // a read of this block, or half of the next ones' copies and reads
            constexpr int CP = h < 0 ? 0 : Cfg::LOADS / 2, OPS = h < 0 ? 1 : CP + 1 + JT / 2;
            static_assert(Cfg::LOADS % 2 == 0 && JT % 2 == 0, "halves");
            each<N>([&](auto M) {
                constexpr int n = decltype(M)::value, k = n / JT, j = n % JT;
                each<OPS>([&](auto O) {
                    constexpr int o = decltype(O)::value, next = h * (JT / 2) + o - CP - 1;
                    if constexpr (o * N / OPS == n) {
                        __builtin_amdgcn_sched_barrier(0);
                        if constexpr (h < 0)
                            p[i & 1] = read_p(kb, i + 2);
                        else if constexpr (o < CP)
                            stage(kb + S, h * CP + o);
                        else if constexpr (o == CP)
                            np[h] = read_p(kb + 1, h);
                        else
                            nxt[next] = read_q(kb + 1, next);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                });
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.k[k], cur[j].k[k], acc[i][j], 0, 0, 0);
            });
        });
        p[0] = np[0];
        p[1] = np[1];
    };
    for (int kb = 0; kb < KB; kb += 2) {   // KB is even: K is a multiple of 128
        block(kb, q[0], q[1]);
        block(kb + 1, q[1], q[0]);
    }
    __builtin_amdgcn_s_waitcnt(0);   // the idle copies have landed,
    __syncthreads();                 // everyone's, and the stages are read out

    // Epilogue.  acc[i][j][r] of lane l is tile row (wm IT + i) 16 + 4 (l / 16)
    // + r, tile column (wn JT + j) 16 + l % 16.  The result is addressed
    // [tile column][tile row] and, transposed, [tile row][tile column].  Written
    // straight from this layout every store would touch 32 bytes of a row (2-byte
    // stores for one of the two), which took as long as the K loop itself; instead
    // each wave turns 16 tile columns at a time through LDS of its own,
    // so that a lane holds 8 consecutive elements of RG rows of the result, and
    // collects 32 tile columns of the transpose in another part, whose rows leave
    // as 64 bytes each.  Both are swizzled against bank conflicts.
    constexpr int SPAN = Cfg::SPAN;        // elements of a result row per wave
    constexpr int LR = SPAN / 8;           // lanes per row
    constexpr int RG = 16 * LR / 64;       // rows per lane
    uint8_t *own = lds + wave * 2 * Cfg::TURN;
    float *strip = reinterpret_cast<float *>(own);                 // [16][SPAN]
    uint8_t *turn = own + Cfg::TURN;                                    // [SPAN][32] FP16 / BF16
    const int rl = lane % LR, rg = lane / LR;                      // element group and row group
    const int e0 = m0 + wm * SPAN + 8 * rl;                        // first element of this lane
    const float inv = 1.0f / kScaleA;
    const int64_t ld_out = MODE == NS_UPDATE ? Np : Mp;
    const float unscale = 1.0f / s;
    const bool mirror = MODE == NS_UPDATE ? last && tall : tc >= (tr + 1) * (TM / TN);
#pragma unroll
    for (int j = 0; j < JT; j++) {
        const int row0 = n0 + (wn * JT + j) * 16 + RG * rg;
        v8h hi[RG], lo[RG];
        if constexpr (MODE == NS_UPDATE) {
#pragma unroll
            for (int q = 0; q < RG; q++) {
                hi[q] = *reinterpret_cast<const v8h *>(xin + (row0 + q) * ld_out + e0);
                const v8h *xl = reinterpret_cast<const v8h *>(xlow + (row0 + q) * ld_out + e0);
                lo[q] = Cfg::STREAM ? __builtin_nontemporal_load(xl) : *xl;
            }
        } else if constexpr (MODE == NS_POLY) {
#pragma unroll
            for (int q = 0; q < RG; q++)
                hi[q] = *reinterpret_cast<const v8h *>(ma + (row0 + q) * ld_out + e0);
        }
#pragma unroll
        for (int i = 0; i < IT; i++) {
            const int c = lane & 15, chunk = (i * 4 + (lane >> 4)) ^ c;
            *reinterpret_cast<v4f *>(strip + (c * SPAN + (chunk & (SPAN / 4 - 1)) * 4)) = acc[i][j];
        }
        // the wave's own LDS accesses are in order; the fence only holds the compiler
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        uint16_t out[RG][8];
#pragma unroll
        for (int q = 0; q < RG; q++) {
            const int c = RG * rg + q, row = row0 + q;
            float v[8];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const v4f w = *reinterpret_cast<const v4f *>(
                    strip + (c * SPAN + (((2 * rl + h) ^ c) & (SPAN / 4 - 1)) * 4));
#pragma unroll
                for (int k = 0; k < 4; k++)
                    v[4 * h + k] = w[k];
            }
            v8h res;
            if constexpr (MODE == NS_GRAM) {
                const float is = kScaleA * unscale * unscale;
#pragma unroll
                for (int k = 0; k < 8; k++)
                    res[k] = (_Float16)as_f32(v[k] * is);
            } else if constexpr (MODE == NS_POLY) {
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float y = as_f32(fmaf(gb, (float)hi[q][k], gc * inv * v[k]));
                    if (e0 + k == row)
                        diag[row] = y;
                    res[k] = (_Float16)(e0 + k == row ? 0.0f : y);
                }
            } else {
                const float f = fmaf(diag[row], inv, ga);
                v8h low;
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    v[k] = as_f32(fmaf(f, (float)hi[q][k] + (float)lo[q][k], v[k] * inv));
                    res[k] = (_Float16)v[k];
                    low[k] = (_Float16)as_f32(v[k] - (float)res[k]);
                }
                if (!last) {
                    v8h *xl = reinterpret_cast<v8h *>(xlow + row * ld_out + e0);
                    if constexpr (Cfg::STREAM)
                        __builtin_nontemporal_store(low, xl);
                    else
                        *xl = low;
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        w[k] = to_bf16x2(v[2 * k] * unscale, v[2 * k + 1] * unscale);
                    if (!tall && row < M)
                        store_run(result + row * ldo, e0, N, w);
                    res = __builtin_bit_cast(v8h, make_uint4(w[0], w[1], w[2], w[3]));
                }
            }
            if (MODE != NS_UPDATE || !last) {
                uint16_t *to = MODE == NS_GRAM ? ma : MODE == NS_POLY ? mb : xout;
                *reinterpret_cast<v8h *>(to + row * ld_out + e0) = res;
            }
            const uint4 bits = __builtin_bit_cast(uint4, res);
            const uint32_t w[4] = {bits.x, bits.y, bits.z, bits.w};
#pragma unroll
            for (int k = 0; k < 8; k++)
                out[q][k] = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
        }
        if (!mirror)
            continue;
        // element 8 rl + k of these RG rows: place k LR + rl of `turn`, 2 RG bytes
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int place = k * LR + rl, byte = (j & 1) * 32 + rg * (2 * RG);
            uint8_t *dst = turn + place * 64 + (byte ^ ((place & 1) << 5));
            if constexpr (RG == 4)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(out[0][k] | ((uint32_t)out[1][k] << 16),
                                                             out[2][k] | ((uint32_t)out[3][k] << 16));
            else if constexpr (RG == 2)
                *reinterpret_cast<uint32_t *>(dst) = out[0][k] | ((uint32_t)out[1][k] << 16);
            else
                *reinterpret_cast<uint16_t *>(dst) = out[0][k];
        }
        if ((j & 1) == 0)
            continue;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int p = 0; p < SPAN / 16; p++) {
            const int place = p * 16 + (lane >> 2), c = lane & 3;
            const int row = m0 + wm * SPAN + 8 * (place % LR) + place / LR;   // of the transpose
            const int col = n0 + (wn * JT + j - 1) * 16 + 8 * c;
            const uint4 w = *reinterpret_cast<const uint4 *>(turn + place * 64 + ((16 * c) ^ ((place & 1) << 5)));
            if constexpr (MODE == NS_UPDATE) {
                const uint32_t o[4] = {w.x, w.y, w.z, w.w};
                if (row < N)
                    store_run(result + row * ldo, col, M, o);
            } else {
                *reinterpret_cast<uint4 *>((MODE == NS_GRAM ? ma : mb) + (int64_t)row * Mp + col) = w;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
}

int pad_to(int n, int t) { return (n + t - 1) / t * t; }

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Lays one matrix out in the workspace from `base` on (NULL: only counts); the bytes used.
size_t lay_out(NsItem &it, char *base)
{
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char *p = base ? base + off : nullptr;
        off += up256(bytes);
        return p;
    };
    const size_t mn = (size_t)it.Mp * it.Np * 2, mm = (size_t)it.Mp * it.Mp * 2;
    it.xh[0] = (uint16_t *)take(mn);
    it.xh[1] = (uint16_t *)take(mn);
    it.xl = (uint16_t *)take(mn);
    it.a = (uint16_t *)take(mm);
    it.b = (uint16_t *)take(mm);
    it.d = (float *)take((size_t)it.Mp * 4);
    it.part = (double *)take(kNormBlocks * sizeof(double));
    return off;
}

NsItem make_item(const NsMatrix &m)
{
    NsItem it;
    it.g = m.g;
    it.o = m.o;
    it.ldg = m.ldg;
    it.ldo = m.ldo;
    it.tall = m.rows > m.cols;
    it.M = (int)std::min(m.rows, m.cols);
    it.N = (int)std::max(m.rows, m.cols);
    it.Mp = pad_to(it.M, 128);
    it.Np = pad_to(it.N, 128);
    it.s = (float)std::exp2(std::round(0.5 * std::log2((double)it.N)));
    return it;
}

template <class Cfg, int MODE> bool fits(const NsItem &it)
{
    return it.Mp % Cfg::TN == 0 && (MODE == NS_UPDATE ? it.Np : it.Mp) % Cfg::TM == 0;
}

template <class Cfg, int MODE> int tiles_of(const NsItem &it)
{
    const int rows = (MODE == NS_UPDATE ? it.Np : it.Mp) / Cfg::TM, cols = it.Mp / Cfg::TN;
    // on and above the diagonal: less the tiles wholly below it
    return rows * cols - (MODE == NS_UPDATE ? 0 : Cfg::TM / Cfg::TN * (rows * (rows - 1) / 2));
}

template <int MODE> int depth_of(const NsItem &it) { return (MODE == NS_GRAM ? it.Np : it.Mp) / 64; }

// Estimated time of a product on Cfg's tiles, us: a fixed part, and the K blocks
// of the busiest of the 256 CUs (the items are sorted, deepest first) times what
// a block takes with at most a tile on every CU (`one`) or more (`many`).
template <class Cfg, int MODE> double estimate(const NsGroup &g, double fixed, double one, double many)
{
    double n = 0, work = 0, most = 0;
    for (int i = 0; i < g.count; i++) {
        if (!fits<Cfg, MODE>(g.it[i]))
            return 1e30;
        const double t = tiles_of<Cfg, MODE>(g.it[i]), k = depth_of<MODE>(g.it[i]);
        n += t;
        work += t * k;
        most = std::max(most, std::ceil(n / 256) * k);
    }
    return fixed + std::max(most, work / 256) * (n <= 256 ? one : many);
}

// first[] from the items' workgroup counts; the launch's number of workgroups.
template <class Count> unsigned deal(NsGroup &g, Count count)
{
    int n = 0;
    for (int i = 0; i <= kNsGroupMax; i++) {
        g.first[i] = i <= g.count ? n : INT_MAX;
        n += i < g.count ? count(g.it[i]) : 0;
    }
    return (unsigned)n;
}

template <class Cfg, int MODE> hipError_t launch_tiles(NsGroup &g, hipStream_t st)
{
    const unsigned n = deal(g, tiles_of<Cfg, MODE>);
    hipLaunchKernelGGL((ns_product_kernel<Cfg, MODE>), dim3(n), dim3(Cfg::THREADS), 0, st, g);
    return hipGetLastError();
}

// One product of every matrix, the deepest first: their tiles take longest.
// The block times are measured on a busy GPU; what they choose is the fastest of
// the four in all of these (us, with 256 x 256, 256 x 128, 128 x 128 and 64 x 64
// tiles): X X^T of one 1024 x 1024 matrix 28, 17, 11 and 8, one 1024 x 4096 74, 43,
// 25 and 16, one 2048 x 2048 44, 26, 19 and 24, two of them 45, 29, 37 and 40, a
// layer's seven gradients 147, 117, 129 and 210; B X of one 2048 x 2048 51, 33, 26
// and 35, two of them 55, 42, 47 and 62, a layer's 205, 252, 283 and 381.
template <int MODE> hipError_t launch_product(NsGroup &g, hipStream_t st)
{
    std::stable_sort(g.it, g.it + g.count,
                     [](const NsItem &x, const NsItem &y) { return depth_of<MODE>(x) > depth_of<MODE>(y); });
    const double l = estimate<NsL, MODE>(g, 7.0, 1.47, 1.47), m = estimate<NsM, MODE>(g, 6.0, 0.8, 1.05),
                 q = estimate<NsQ, MODE>(g, 4.5, 0.48, 0.63), e = estimate<NsE, MODE>(g, 3.8, 0.2, 0.3);
    const double best = std::min(std::min(l, m), std::min(q, e));
    if (best == l)
        return launch_tiles<NsL, MODE>(g, st);
    if (best == m)
        return launch_tiles<NsM, MODE>(g, st);
    return best == q ? launch_tiles<NsQ, MODE>(g, st) : launch_tiles<NsE, MODE>(g, st);
}

hipError_t launch_step(NsGroup &g, hipStream_t st)
{
    hipError_t e = launch_product<NS_GRAM>(g, st);
    if (e == hipSuccess)
        e = launch_product<NS_POLY>(g, st);
    if (e == hipSuccess)
        e = launch_product<NS_UPDATE>(g, st);
    return e;
}

} // namespace

// Matrices of one call run kNsGroupMax at a time; the groups follow each other
// on the stream and share the workspace.
size_t newton_workspace_bytes(const NsMatrix *ms, int count)
{
    size_t most = 0;
    for (int lo = 0; lo < count; lo += kNsGroupMax) {
        size_t sum = 0;
        for (int i = lo; i < std::min(count, lo + kNsGroupMax); i++) {
            NsItem it = make_item(ms[i]);
            sum += lay_out(it, nullptr);
        }
        most = std::max(most, sum);
    }
    return most;
}

hipError_t launch_newton(const NsMatrix *ms, int count, bool gbf16, int steps, const float *coef, float eps,
                         void *workspace, hipStream_t st)
{
    for (int lo = 0; lo < count; lo += kNsGroupMax) {
        NsGroup g;
        g.count = std::min(count - lo, kNsGroupMax);
        g.gbf16 = gbf16;
        g.eps = eps;
        size_t off = 0;
        for (int i = 0; i < g.count; i++) {
            g.it[i] = make_item(ms[lo + i]);
            off += lay_out(g.it[i], (char *)workspace + off);
        }
        hipLaunchKernelGGL(ns_norm_kernel, dim3(kNormBlocks, (unsigned)g.count), dim3(256), 0, st, g);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess)
            return e;
        const unsigned n = deal(g, [](const NsItem &it) { return (it.Mp / 64) * (it.Np / 64); });
        hipLaunchKernelGGL(ns_init_kernel, dim3(n), dim3(256), 0, st, g);
        e = hipGetLastError();
        for (int k = 0; k < steps && e == hipSuccess; k++) {
            g.a = coef[3 * k];
            g.b = coef[3 * k + 1];
            g.c = coef[3 * k + 2];
            g.last = k + 1 == steps;
            e = launch_step(g, st);
            for (int i = 0; i < g.count; i++)
                std::swap(g.it[i].xh[0], g.it[i].xh[1]);
        }
        if (e != hipSuccess)
            return e;
    }
    return hipSuccess;
}

} // namespace puro
