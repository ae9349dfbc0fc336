/*
 * fp4_layer.h -- C ABI of libfp4, layer operators around the 8-bit floating-point
 * products: the root-mean-square norm and the SwiGLU that write 8-bit activations with
 * their scales, the product whose two operands carry a scale per block of 128, the
 * routing of tokens to experts, and the experts' products.
 *
 * The conventions of fp4.h hold (device pointers, caller-owned memory, asynchronous on
 * `stream`, no allocation, no synchronisation, host checks before any launch, thread
 * safety, status codes, fp4_last_error), with these additions:
 *   - FP8 grids only: fp4_grid E4M3 (e = 4, m = 3) or E5M2 (e = 5, m = 2), one code per
 *     byte.
 *   - Granularities are fp4_gran's; here a GROUP need not divide the row: the last group
 *     of a row is the shorter one, and a row has ceil(cols / group) scales.
 *   - Rows are read and written 16 bytes (codes: 8 bytes) at a time: element pointers are
 *     16-byte aligned, leading dimensions are multiples of 16 bytes (codes: of 8 bytes),
 *     and the number of columns is a multiple of 8.
 *   - Outputs may not overlap inputs, except where a call says so.
 *   - Work whose threads would pass 2^32, the most one launch takes, is split over launches.
 */
#ifndef FP4_LAYER_H_
#define FP4_LAYER_H_

#include "fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- residual addition, root-mean-square norm, 8-bit output ---------------------- */
typedef struct {
    int64_t rows, cols;         /* cols <= 65536, a multiple of 8                     */
    const void* x;              /* [rows * terms, cols], leading dim ldx              */
    int64_t ldx;                /* elements                                           */
    int32_t x_dtype;            /* FP4_F32 or FP4_BF16                                */
    int32_t terms;              /* rows of x added into each row of the stream, 1..64 */
    const float* term_weights;  /* f32 [rows, terms] contiguous, or NULL (all 1)      */
    const void* residual;       /* [rows, cols], leading dim ldr, or NULL (zero)      */
    int64_t ldr;
    void* residual_out;         /* [rows, cols], leading dim ldro, or NULL: the summed
                                   stream; may be `residual` itself (same ld)         */
    int64_t ldro;
    int32_t residual_dtype;     /* FP4_F32 or FP4_BF16, of both                       */
    int32_t gamma_dtype;        /* FP4_F32 or FP4_BF16                                */
    const void* gamma;          /* [cols]                                             */
    float eps;                  /* >= 0                                               */
    int32_t y_dtype;            /* FP4_F32 or FP4_BF16                                */
    void* y;                    /* [rows, cols], leading dim ldy, or NULL: the normed
                                   rows themselves (a router's input)                 */
    int64_t ldy;
    fp4_grid grid;
    fp4_gran gran;              /* ROW, GROUP, or TENSOR with tensor_scale            */
    const float* tensor_scale;  /* TENSOR: the f32 scale s                            */
    const int8_t* col_shift;    /* TENSOR: int8 k[cols] in [-64, 0], or NULL          */
    uint8_t* packed;            /* codes [rows, cols], leading dim ldp bytes, or NULL */
    int64_t ldp;
    void* scales;               /* ROW / GROUP: f32 or f16 per unit, as gran says     */
} fp4_rmsnorm_desc;

/* For every row r:
 *   h = residual[r] + sum_j w[r, j] x[r * terms + j]   (j in order, one fused multiply-
 *       add each; w = 1 without term_weights).  A term whose weight is 0 is absent: its
 *       row of x is read as zeros whatever it holds.
 *   n = (h / sqrt(mean(h^2) + eps)) * gamma, everything in binary32
 *   residual_out = h, y = n, each rounded to its type
 *   codes of n: per unit (row or group) s = fl32(amax / Qmax), no less than 2^-126 unless
 *       amax is 0 (rounded to binary16 for f16 scales), codes of fl32(n * fl32(1/s)) as
 *       fp4_quantize_pack; with TENSOR the given scale and shifts, codes of
 *       fl32(n * fl32(1/s) 2^-k), a factor past binary32 being its largest number.  Zeros
 *       have the codes of zero whatever the scale.
 * At least one of packed, y, residual_out is given.  Several terms are an expert layer's
 * outputs (one row per token and chosen expert, fp4_route's weights) joining the stream. */
fp4_status fp4_rmsnorm_quant(const fp4_rmsnorm_desc* d, void* stream);

/* ---- SwiGLU with 8-bit output ----------------------------------------------------- */
typedef struct {
    int64_t rows, cols;         /* of the output; cols <= 65536, a multiple of 8      */
    const void* x;              /* [rows, 2 cols]: gate columns, then up columns      */
    int64_t ldx;                /* elements                                           */
    int32_t x_dtype;            /* FP4_F32 or FP4_BF16                                */
    int32_t reserved;           /* must be 0                                          */
    fp4_grid grid;
    fp4_gran gran;              /* as fp4_rmsnorm_desc                                */
    const float* tensor_scale;
    const int8_t* col_shift;
    uint8_t* packed;            /* codes [rows, cols], leading dim ldp bytes          */
    int64_t ldp;
    void* scales;
} fp4_swiglu8_desc;

/* h = (g / (1 + e^-g)) u in binary32, g = x[:, 0:cols], u = x[:, cols:2 cols]; codes and
 * scales of h as fp4_rmsnorm_quant's of n.  e^-g is 2^(-g log2 e), it and the reciprocal are
 * the hardware's: h is within (2 |g| + 8) 2^-24 of its exact value, relative, and within
 * 2^-100 |u| for gates below -87, where e^-g may overflow. */
fp4_status fp4_swiglu_quant(const fp4_swiglu8_desc* d, void* stream);

/* ---- weights with a scale per block of 128 x 128 ---------------------------------- */
/* For each of `batch` matrices w[b] = w + b * stride_w elements, [n, k] with leading dim
 * ldw: every block of 128 rows and 128 columns (the last ones shorter) gets
 * s = fl32(amax / Qmax), no less than 2^-126 unless amax is 0, and the codes of
 * fl32(w * fl32(1/s)).
 *   w_dtype  FP4_F32 or FP4_BF16; k a multiple of 8
 *   packed   codes [batch][n, k], leading dim ldp bytes, matrices stride_p bytes apart, none of
 *            which share a byte (those of w may)
 *   scales   f32 [batch, ceil(n / 128), ceil(k / 128)] contiguous                     */
fp4_status fp4_quantize_block(const void* w, int32_t w_dtype, int64_t batch, int64_t n, int64_t k,
                              int64_t ldw, int64_t stride_w, fp4_grid grid, uint8_t* packed,
                              int64_t ldp, int64_t stride_p, float* scales, void* stream);

/* ---- product of 8-bit operands with block scales ---------------------------------- */
typedef struct {
    int64_t M, N, K;            /* Y [M, N] = X [M, K] W [N, K]^T; K a multiple of 16  */
    const uint8_t* a;           /* codes [M, K], leading dim lda bytes (multiple of 16) */
    int64_t lda;
    const float* a_scales;      /* f32 [M, ceil(K / 128)], leading dim lda_s           */
    int64_t lda_s;
    fp4_grid a_grid;
    const uint8_t* w;           /* codes [N, K], leading dim ldw bytes (multiple of 16) */
    int64_t ldw;
    const float* w_scales;      /* f32 [ceil(N / 128), ceil(K / 128)], leading dim ldw_s */
    int64_t ldw_s;
    fp4_grid w_grid;
    void* y;                    /* [M, N], leading dim ldy elements (any >= N)         */
    int64_t ldy;
    int32_t y_dtype;            /* FP4_BF16 or FP4_F32                                 */
    int32_t reserved;           /* must be 0                                           */
} fp4_gemm_block_desc;

/* Y[m, n] = T,  T = sum over the blocks b of 128 columns of K, in order, of
 *   T = fma(P_b[m, n], fl32(a_scales[m, b] * w_scales[n / 128, b]), T),
 * P_b the block's sum of code products on the f8f6f4 matrix cores in binary32 (within
 * fp4_gemm's W8A8 tolerance of the exact value); small products may be summed as several
 * parts of K (ranges, or every so many blocks) that are then added in order.  The result
 * does not depend on timing; which parts depends on the sizes.
 * Rows of a and w shorter than 4 MiB (lda, ldw), else FP4_ERR_UNSUPPORTED. */
fp4_status fp4_gemm_block(const fp4_gemm_block_desc* d, void* stream);

/* ---- routing of tokens to experts -------------------------------------------------- */
#define FP4_ROUTE_SOFTMAX 0
#define FP4_ROUTE_SIGMOID 1
typedef struct {
    int64_t tokens;             /* tokens * top_k < 2^31                              */
    int32_t experts;            /* 1..1024                                            */
    int32_t top_k;              /* 1..32, <= experts                                  */
    const void* logits;         /* [tokens, experts], leading dim ld (any >= experts) */
    int64_t ld;                 /* elements                                           */
    int32_t logits_dtype;       /* FP4_F32 or FP4_BF16 (element-aligned)              */
    int32_t score;              /* FP4_ROUTE_SOFTMAX or FP4_ROUTE_SIGMOID             */
    const float* bias;          /* f32 [experts] added for the choice only, or NULL;
                                   -inf or NaN: no token may choose the expert        */
    int32_t groups;             /* experts form this many equal groups (1: none), <= 64 */
    int32_t top_groups;         /* groups a token may use, 1..groups                  */
    int32_t group_top;          /* a group's value: the sum of its best 1 or 2 keys   */
    int32_t renormalise;        /* nonzero: weights divided by their sum              */
    float scale;                /* factor of every weight                             */
    int32_t reserved;           /* must be 0                                          */
    int32_t* experts_out;       /* int32 [tokens, top_k]                              */
    float* weights_out;         /* f32 [tokens, top_k]                                */
    int32_t* offsets;           /* int32 [experts + 1], or NULL with slots            */
    int32_t* slots;             /* int32 [tokens * top_k], or NULL with offsets       */
} fp4_route_desc;

/* Workspace bytes that fp4_route's layout needs for these sizes (0 for few tokens). */
size_t fp4_route_workspace_size(int64_t tokens, int32_t experts, int32_t top_k);

/* For every token t, over its usable experts -- those whose logit is finite; infinite
 * (either sign) and NaN logits mark experts the token may not use:
 *   score = softmax over the usable logits, or 1 / (1 + e^-logit); binary32.  (An expert
 *     whose bias is -inf or NaN has a score, and counts in the softmax, but none of what
 *     follows chooses it; a bias of +inf comes first.)
 *   groups > 1: a group's value is the sum of its group_top largest score + bias (of fewer,
 *     if fewer are usable); only experts of the top_groups best groups that have a usable
 *     expert stay (ties: the lower group)
 *   experts_out[t] = the top_k best by score + bias -- without a bias by the logit itself,
 *     which has the scores' order and neither rounds nor underflows -- best first, ties to
 *     the lower index; a token with fewer stays short: expert -1 with weight 0
 *   weights_out[t] = the scores (without bias) of those, divided by their sum with
 *     `renormalise` (a sum of 0 leaves 0), times `scale`; the exponential and the reciprocal
 *     are the hardware's: a weight is within (2 d + 40) 2^-24 of its exact value, relative, d the
 *     largest distance of the token's usable logits from their largest (softmax) or from 0
 * Layout (offsets and slots given): slot t * top_k + j belongs to experts_out[t, j];
 * slots holds all slot numbers ordered by expert and, within an expert, ascending, expert
 * e's at offsets[e] .. offsets[e + 1]; the slots of expert -1 follow offsets[experts].
 *   workspace  device scratch of at least fp4_route_workspace_size() bytes            */
fp4_status fp4_route(const fp4_route_desc* d, void* workspace, size_t ws_bytes, void* stream);

/* ---- the experts' products ---------------------------------------------------------- */
typedef struct {
    int64_t slots;              /* rows of Y; < 2^31 - 2^18                           */
    int64_t N, K;               /* of each expert; K a multiple of 16                 */
    int32_t experts;            /* 1..1024                                            */
    int32_t slots_per_row;      /* slot s reads row s / slots_per_row of a: top_k for
                                   one row per token, 1 for one row per slot          */
    const uint8_t* a;           /* codes [ceil(slots / slots_per_row), K], leading dim lda */
    int64_t lda;                /* bytes, multiple of 16                              */
    const float* a_scales;      /* f32, a row per row of a, leading dim lda_s         */
    int64_t lda_s;
    fp4_grid a_grid;
    const uint8_t* w;           /* codes [experts][N, K], leading dim ldw bytes       */
    int64_t ldw, stride_w;      /* stride_w: bytes between experts (multiples of 16)  */
    const float* w_scales;      /* f32 [experts, ceil(N / 128), ceil(K / 128)] contiguous */
    fp4_grid w_grid;
    const int32_t* offsets;     /* fp4_route's layout (device)                        */
    const int32_t* slot_list;   /* fp4_route's slots (device), `slots` entries        */
    void* y;                    /* [slots, N], leading dim ldy elements               */
    int64_t ldy;
    int32_t y_dtype;            /* FP4_BF16 or FP4_F32                                */
    int32_t reserved;           /* must be 0                                          */
} fp4_gemm_experts_desc;

/* Y[s] = X[s / slots_per_row] W[e]^T for every slot s in slot_list[offsets[e] ..
 * offsets[e + 1]), with fp4_gemm_block's definition of the product.  Rows of slots that
 * no expert holds are not written.  Offsets are read as limited to [0, slots] and slot
 * numbers outside [0, slots) are skipped.  a spans less than 2 GiB (lda times its rows),
 * rows of w less than 4 MiB, else FP4_ERR_UNSUPPORTED. */
fp4_status fp4_gemm_experts(const fp4_gemm_experts_desc* d, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4_LAYER_H_ */
