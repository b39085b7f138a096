// Internal launchers (host side).  Arguments are validated by the C-ABI layer
// before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stddef.h>

namespace puro {

// pow2: power-of-two block scales (the scaled matrix cores' E8M0 variant)
// instead of amax / 448.
hipError_t launch_quant_act(const void *x, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                            uint8_t *q, int64_t ldq, float *s, bool pow2, hipStream_t st);
hipError_t launch_quant_weight(const void *w, bool bf16, int64_t rows, int64_t cols, int64_t ldw,
                               uint8_t *q, int64_t ldq, float *s, bool pow2, hipStream_t st);
// One weight of a grouped weight quantisation (as launch_quant_weight's
// arguments; cb = number of 128-column tiles).
struct QuantWeightItem {
    const void *w;
    int64_t rows, cols, ldw;
    uint8_t *q;
    int64_t ldq;
    float *s;
    int64_t cb;        // ceil(cols / 128)
    uint8_t *qt;       // transposed codes [cols][rows] (row stride ldqt), or NULL
    int64_t ldqt;
    float *st;         // transposed scales [cb][rb], dense (with qt)
    int64_t rb;        // ceil(rows / 128)
};
constexpr int kQuantGroupMax = 16;   // weights per launch; more take several launches
hipError_t launch_quant_weight_group(const QuantWeightItem *items, int count, bool bf16, bool pow2,
                                     hipStream_t st);
hipError_t launch_quant_transpose(const void *x, bool bf16, int64_t tokens, int64_t cols,
                                  int64_t ldx, bool transpose_out, uint8_t *q, int64_t ldq,
                                  float *s, bool pow2, hipStream_t st);
hipError_t launch_quant_dual(const void *x, bool bf16, int64_t tokens, int64_t cols, int64_t ldx,
                             uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                             int64_t ldqt, float *st, bool pow2, hipStream_t stream);

// Dual quantiser of h = BF16(silu(g) * u), g and u BF16 [tokens][cols]; h is
// also stored unless NULL.
hipError_t launch_swiglu_dual(const uint16_t *g, int64_t ldg, const uint16_t *u, int64_t ldu, uint16_t *h,
                              int64_t ldh, int64_t tokens, int64_t cols, uint8_t *qr, int64_t ldqr, float *sr,
                              bool transpose_out, uint8_t *qt, int64_t ldqt, float *st, bool pow2,
                              hipStream_t stream);

// Norm: z = BF16(x + res) (x itself when res is NULL, and z unused), r = 1 /
// sqrt(mean z^2 + eps) to rstd, n = z r w.  h: BF16(n) is stored there unless NULL.
struct NormIn {
    const uint16_t *x;
    int64_t ldx;
    const uint16_t *res;
    int64_t ldres;
    const void *w;
    bool wbf16;
    float eps;
    int64_t tokens, cols;
    uint16_t *z;
    int64_t ldz;
    float *rstd;   // may be NULL in launch_norm_act
    uint16_t *h;
    int64_t ldh;
};
hipError_t launch_norm_act(const NormIn &in, uint8_t *q, int64_t ldq, float *s, bool pow2, hipStream_t st);
hipError_t launch_norm_dual(const NormIn &in, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                            int64_t ldqt, float *stok, bool pow2, hipStream_t st);

// Norm gradient: dx = dres + r (w dy - z r mean(w dy z r)) (dres may be NULL),
// dw = (dw +) sum over tokens of dy z r.
struct NormBwd {
    const uint16_t *dy;
    int64_t lddy;
    const uint16_t *z;
    int64_t ldz;
    const float *rstd;
    const void *w;
    bool wbf16;
    const uint16_t *dres;
    int64_t lddres;
    int64_t tokens, cols;
    uint16_t *dx;
    int64_t lddx;
    float *dw;
    bool accumulate;
};
size_t norm_bwd_workspace_bytes(int64_t tokens, int64_t cols);
hipError_t launch_norm_bwd(const NormBwd &b, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt,
                           int64_t ldqt, float *stok, bool pow2, void *workspace, hipStream_t st);

// Gradient of h = silu(g) u, both halves quantised both ways.
struct GradOut {
    uint8_t *q_row;
    int64_t ldq_row;
    float *s_row;
    int64_t lds_row;   // row strides of the scale arrays
    uint8_t *q_tok;
    int64_t ldq_tok;
    float *s_tok;
    int64_t lds_tok;
};
struct SwigluBwd {
    const uint16_t *dh;
    int64_t lddh;
    const uint16_t *g;
    int64_t ldg;
    const uint16_t *u;
    int64_t ldu;
    int64_t tokens, cols;
    GradOut dgate, dup;
};
hipError_t launch_swiglu_bwd(const SwigluBwd &b, bool transpose_out, bool pow2, hipStream_t st);

// Newton-Schulz orthogonalisation of `count` matrices [rows][cols] (FP32 or
// BF16), results in BF16; coef holds a, b, c of every step.
struct NsMatrix {
    const void *g;
    int64_t rows, cols, ldg;
    void *o;
    int64_t ldo;
};
constexpr int kNsGroupMax = 16;   // matrices per launch; more take several rounds
size_t newton_workspace_bytes(const NsMatrix *ms, int count);
hipError_t launch_newton(const NsMatrix *ms, int count, bool gbf16, int steps, const float *coef, float eps,
                         void *workspace, hipStream_t st);

// Norm of query and key heads (none when wq is NULL) and rotation of the first `rotary` elements of each.
struct RopeShape {
    const uint16_t *q;
    int64_t ldq;
    const uint16_t *k;
    int64_t ldk;
    int hq, hk, dim;   // 64 or 128 elements a head
    int64_t tokens;
    const void *wq, *wk;
    bool wbf16;
    float eps;
    const int32_t *pos;    // [tokens]
    const float *freq;     // [rotary / 2]
    int rotary;            // a multiple of 16
    float mscale;
    bool interleaved;      // pairs (2 j, 2 j + 1) instead of (j, j + rotary / 2)
};
// parts (waves a token's heads are spread over), turn and part are the launchers'.
struct RopeFwd {
    RopeShape r;
    uint16_t *qo;
    int64_t ldqo;
    uint16_t *ko;
    int64_t ldko;
    float *rstd;           // [tokens][hq + hk], or NULL
    int parts;
};
hipError_t launch_rope(RopeFwd a, hipStream_t st);
struct RopeBwd {
    RopeShape r;
    const uint16_t *dq;
    int64_t lddq;
    const uint16_t *dk;
    int64_t lddk;
    const uint16_t *dv;
    int64_t lddv;
    const float *rstd;
    uint16_t *dx;          // joint gradient in BF16, or NULL
    int64_t lddx;
    float *dwq, *dwk;
    bool accumulate;
    const float2 *turn;    // [tokens][rotary / 2]
    float *part;           // [token tile][(hq + hk) dim]
};
size_t rope_bwd_workspace_bytes(const RopeShape &r, bool norm);
hipError_t launch_rope_bwd(RopeBwd b, uint8_t *qr, int64_t ldqr, float *sr, bool transpose_out, uint8_t *qt, int64_t ldqt,
                           float *stok, bool pow2, void *workspace, hipStream_t st);

// Attention of packed sequences: sequence s's query rows are q_off[s] .. and its key rows k_off[s] .., len[s] of
// them (up to the next offset where len is NULL; all arrays in device memory).
struct AttnShape {
    int hq, hk, dim;   // query heads, key heads (hq a multiple), 64 or 128 elements each
    int seqs;
    const int32_t *q_off, *q_len, *k_off, *k_len;
    int64_t tokens_q, tokens_k;
    int max_q, max_k;  // no sequence's rows count past these
    bool causal;
};
// c2, splits, blocks and the pointers into the workspace are the launchers'.
struct AttnFwd {
    AttnShape s;
    const uint16_t *q;
    int64_t ldq;
    const uint16_t *k;
    int64_t ldk;
    const uint16_t *v;
    int64_t ldv;
    float scale;
    uint16_t *o;
    int64_t ldo;
    float *lse;        // [hq][tokens_q], or NULL
    float c2;
    int splits, blocks;
    float *part;       // [split][hq][tokens_q][dim]
    float2 *stat;      // [split][hq][tokens_q]: maximum (log2 units), sum
};
// Whether every launch's work items fit the 32 bits that a grid has.
bool attn_fits(const AttnShape &s, bool backward);
size_t attn_workspace_bytes(const AttnShape &s);
hipError_t launch_attn(AttnFwd a, void *workspace, hipStream_t st);

struct AttnBwd {
    AttnShape s;
    const uint16_t *dout;
    int64_t lddo;
    const uint16_t *q;
    int64_t ldq;
    const uint16_t *k;
    int64_t ldk;
    const uint16_t *v;
    int64_t ldv;
    const uint16_t *o;
    int64_t ldo;
    const float *lse;
    float scale;
    uint16_t *dq;
    int64_t lddq;
    uint16_t *dk;
    int64_t lddk;
    uint16_t *dv;
    int64_t lddv;
    float c2;
    int q_blocks;
    float *nl, *nd;    // [hq][tokens_q]: -lse / scale, -D (sum of do o, or of P dP for rows that see few keys)
};
size_t attn_bwd_workspace_bytes(const AttnShape &s);
hipError_t launch_attn_bwd(AttnBwd b, void *workspace, hipStream_t st);

constexpr int kGemmMaxSeg = 4;

// One K segment of a product: A, B and their block scales over K indices 0 .. K-1.
struct GemmSegment {
    int64_t K;
    const uint8_t *A;
    int64_t lda;
    const float *sA;
    const uint8_t *B;
    int64_t ldb;
    const float *sB;
};

// C (+)= sum over segments of the blockwise product; the segments share M, N
// and the output.
struct GemmProblem {
    int layout;   // 0 NT, 1 NN, 2 TN
    int bgran;    // 0 1x128, 1 128x128
    bool c_bf16;  // output dtype
    bool accumulate;
    int64_t M, N;
    int nseg;
    GemmSegment seg[kGemmMaxSeg];
    void *C;
    int64_t ldc;
};

// Single-segment, overwriting problems (accumulate and extra segments are the
// grouped launcher's).
size_t gemm_workspace_bytes(const GemmProblem &p);
hipError_t launch_gemm(const GemmProblem &p, void *workspace, hipStream_t st);
// Scaled-matrix-core variant: power-of-two scales, M, N, K multiples of 128.
size_t gemm_mx_workspace_bytes(const GemmProblem &p);
hipError_t launch_gemm_mx(const GemmProblem &p, void *workspace, hipStream_t st);
// Native FP8 matrix-core variant: amax/448 scales as in launch_gemm, block
// partials on the FP8 matrix cores (not FP32-exact), M, N, K multiples of 128.
size_t gemm_native_workspace_bytes(const GemmProblem &p);
hipError_t launch_gemm_native(const GemmProblem &p, void *workspace, hipStream_t st);
// Independent problems sharing layout, B-scale granularity and output dtype;
// needs no workspace.
hipError_t launch_gemm_group(const GemmProblem *probs, int count, hipStream_t st);
// The same on the scaled (MX) and on the native FP8 datapaths: aligned
// problems only (M, N and every segment's K multiples of 128).
hipError_t launch_gemm_group_mx(const GemmProblem *probs, int count, hipStream_t st);
hipError_t launch_gemm_group_native(const GemmProblem *probs, int count, hipStream_t st);

} // namespace puro
