// Host layer of the operators of include/fp4_layer.h: argument validation (before any
// launch) and dispatch to the HIP kernels.
#include "../../include/fp4_layer.h"
#include "layer_internal.h"

using namespace fp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool float_type(int32_t t) { return t == FP4_F32 || t == FP4_BF16; }

int64_t size_of(int32_t t) { return t == FP4_BF16 ? 2 : 4; }

// a * b stays below `limit` (a, b >= 0)
bool below(int64_t a, int64_t b, int64_t limit) { return b == 0 || a <= (limit - 1) / b; }

fp4_status fp8_grid(const fp4_grid& g, QGrid* q) {
    fp4_status st = grid_table(g, q);
    if (st) return st;
    if (q->kind != 0 || q->bits != 8) return report(FP4_ERR_UNSUPPORTED, "the grid must be FP8 E4M3 or E5M2");
    return FP4_OK;
}

// `count` rows or matrices `stride` elements apart (both >= 0) have byte offsets of 64 bits
fp4_status spans(const char* name, int64_t count, int64_t stride) {
    if (!below(count, stride, 1ll << 60)) return report(FP4_ERR_UNSUPPORTED, "%s spans more than 2^60 elements", name);
    return FP4_OK;
}

// the matrix [rows, cols] at p: leading dimension and alignment of 16-byte accesses
fp4_status matrix(const char* name, const void* p, int64_t rows, int64_t ld, int64_t cols, int32_t type) {
    if (ld < cols) return report(FP4_ERR_INVALID_ARG, "leading dimension of %s below its columns", name);
    fp4_status st = spans(name, rows, ld);
    if (st) return st;
    if (!aligned(p, 16) || (ld * size_of(type)) % 16 != 0)
        return report(FP4_ERR_ALIGNMENT, "%s must be 16-byte aligned, its rows a multiple of 16 bytes apart", name);
    return FP4_OK;
}

// codes and scales of rows of `cols` values; *out is filled in
fp4_status code_output(int64_t rows, int64_t cols, const fp4_grid& grid, const fp4_gran& gran, const float* tensor_scale,
                       const int8_t* col_shift, uint8_t* packed, int64_t ldp, void* scales, CodeOut* out) {
    QGrid q;
    fp4_status st = fp8_grid(grid, &q);
    if (st) return st;
    if (gran.reserved != 0) return report(FP4_ERR_INVALID_ARG, "fp4_gran.reserved must be 0");
    if (gran.mode < FP4_SCALE_TENSOR || gran.mode > FP4_SCALE_GROUP)
        return report(FP4_ERR_INVALID_ARG, "bad scale mode %d", gran.mode);
    if (gran.scale_dtype != FP4_F32 && gran.scale_dtype != FP4_F16)
        return report(FP4_ERR_INVALID_ARG, "scale dtype must be FP4_F32 or FP4_F16");
    if (gran.mode == FP4_SCALE_TENSOR) {
        if (gran.scale_dtype != FP4_F32) return report(FP4_ERR_UNSUPPORTED, "per-tensor scales are f32 only");
        if (!tensor_scale) return report(FP4_ERR_UNSUPPORTED, "TENSOR mode needs a given tensor_scale");
    } else {
        if (tensor_scale || col_shift) return report(FP4_ERR_INVALID_ARG, "tensor_scale and col_shift need TENSOR mode");
        if (!scales) return report(FP4_ERR_INVALID_ARG, "scales must be given with ROW and GROUP scales");
    }
    if (gran.mode == FP4_SCALE_GROUP && (gran.group < 8 || gran.group > 512 || (gran.group & (gran.group - 1))))
        return report(FP4_ERR_UNSUPPORTED, "group must be a power of two in [8, 512] (got %d)", gran.group);
    if (ldp < cols) return report(FP4_ERR_INVALID_ARG, "ldp below the code bytes of a row");
    if ((st = spans("packed", rows, ldp))) return st;
    if (!aligned(packed, 8) || ldp % 8 != 0 || !aligned(col_shift, 8))
        return report(FP4_ERR_ALIGNMENT, "packed and col_shift must be 8-byte aligned, ldp a multiple of 8");
    if (!aligned(tensor_scale, 4) || !aligned(scales, gran.scale_dtype == FP4_F16 ? 2 : 4))
        return report(FP4_ERR_ALIGNMENT, "scales must be aligned to their type");
    out->packed = packed;
    out->ldp = ldp;
    out->e4m3 = q.e == 4;
    out->mode = gran.mode;
    out->group = gran.mode == FP4_SCALE_GROUP ? gran.group : 0;
    out->scale_f16 = gran.scale_dtype == FP4_F16;
    out->qmax = q.qmax;
    out->rqmax = 1.0f / q.qmax;
    out->tensor_scale = tensor_scale;
    out->col_shift = col_shift;
    out->scales = scales;
    return FP4_OK;
}

fp4_status row_sizes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > 0x7fffffff) return report(FP4_ERR_INVALID_ARG, "bad sizes rows=%lld cols=%lld",
                                                                 (long long)rows, (long long)cols);
    if (cols % 8 != 0 || cols > 65536)
        return report(FP4_ERR_UNSUPPORTED, "cols must be a multiple of 8, at most 65536 (got %lld)", (long long)cols);
    return FP4_OK;
}

// operand of a block-scaled product: codes [., K] at p
fp4_status code_operand(const char* name, const void* p, int64_t ld, int64_t K, const fp4_grid& grid, int32_t* format) {
    QGrid q;
    fp4_status st = fp8_grid(grid, &q);
    if (st) return st;
    if (ld < K) return report(FP4_ERR_INVALID_ARG, "leading dimension of %s below K", name);
    if (ld >= (1 << 22)) return report(FP4_ERR_UNSUPPORTED, "rows of %s must be shorter than 4 MiB", name);
    if (!aligned(p, 16) || ld % 16 != 0)
        return report(FP4_ERR_ALIGNMENT, "%s must be 16-byte aligned, its rows a multiple of 16 bytes apart", name);
    *format = q.e == 4 ? 0 : 1;
    return FP4_OK;
}

fp4_status product_sizes(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K <= 0 || M > 0x7fffffff || N > 0x7fffffff)
        return report(FP4_ERR_INVALID_ARG, "bad sizes M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
    if (K % 16 != 0) return report(FP4_ERR_UNSUPPORTED, "K must be a multiple of 16 (got %lld)", (long long)K);
    return FP4_OK;
}

fp4_status product_output(const void* y, int64_t M, int64_t ldy, int64_t N, int32_t type) {
    if (!float_type(type)) return report(FP4_ERR_INVALID_ARG, "y_dtype must be FP4_F32 or FP4_BF16");
    if (ldy < N) return report(FP4_ERR_INVALID_ARG, "ldy below N");
    fp4_status st = spans("y", M, ldy);
    if (st) return st;
    if (!aligned(y, 16)) return report(FP4_ERR_ALIGNMENT, "y must be 16-byte aligned");
    return FP4_OK;
}

// whether two of `batch` matrices of n rows of k bytes, rows ld (>= k) and matrices `stride` bytes
// apart, share a byte: rows of matrices i and i + d do if d * stride is less than k from a
// multiple of ld that is below n * ld
bool overlap(int64_t batch, int64_t n, int64_t k, int64_t ld, int64_t stride) {
    const int64_t span = (n - 1) * ld + k;
    if (batch < 2 || stride >= span || (stride >= k && (batch - 1) * stride + k <= ld)) return false;
    for (int64_t d = 1; d < batch && d * stride < span; d++) {
        const int64_t rest = d * stride % ld;
        if (rest < k || (rest > ld - k && d * stride / ld + 1 < n)) return true;
    }
    return false;
}

int64_t blocks_of(int64_t n) { return n / kBlock + (n % kBlock != 0); }

}  // namespace

extern "C" {

fp4_status fp4_rmsnorm_quant(const fp4_rmsnorm_desc* d, void* stream) {
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    fp4_status st = row_sizes(d->rows, d->cols);
    if (st) return st;
    if (d->terms < 1 || d->terms > 64) return report(FP4_ERR_INVALID_ARG, "terms must be 1..64 (got %d)", d->terms);
    if (!float_type(d->x_dtype) || !float_type(d->gamma_dtype) || ((d->residual || d->residual_out) && !float_type(d->residual_dtype)) ||
        (d->y && !float_type(d->y_dtype)))
        return report(FP4_ERR_INVALID_ARG, "element types must be FP4_F32 or FP4_BF16");
    if (!(d->eps >= 0.0f) || d->eps > 3.0e38f) return report(FP4_ERR_INVALID_ARG, "eps must be finite and not negative");
    const bool empty = d->rows == 0 || d->cols == 0;
    if (!d->packed && !d->y && !d->residual_out && !empty) return report(FP4_ERR_INVALID_ARG, "no output is given");
    if (empty) return report_ok();
    if (!d->x || !d->gamma) return report(FP4_ERR_INVALID_ARG, "null pointer");
    NormParams p{};
    if (d->packed && (st = code_output(d->rows, d->cols, d->grid, d->gran, d->tensor_scale, d->col_shift, d->packed, d->ldp, d->scales, &p.out)))
        return st;
    if ((st = matrix("x", d->x, d->rows * d->terms, d->ldx, d->cols, d->x_dtype))) return st;
    if (d->residual && (st = matrix("residual", d->residual, d->rows, d->ldr, d->cols, d->residual_dtype))) return st;
    if (d->residual_out && (st = matrix("residual_out", d->residual_out, d->rows, d->ldro, d->cols, d->residual_dtype))) return st;
    if (d->residual_out && d->residual_out == d->residual && d->ldro != d->ldr)
        return report(FP4_ERR_INVALID_ARG, "residual_out may be residual only with the same leading dimension");
    if (d->y && (st = matrix("y", d->y, d->rows, d->ldy, d->cols, d->y_dtype))) return st;
    if (!aligned(d->gamma, 16) || !aligned(d->term_weights, 4))
        return report(FP4_ERR_ALIGNMENT, "gamma must be 16-byte aligned, term_weights 4-byte aligned");
    p.rows = d->rows;
    p.cols = d->cols;
    p.x = d->x;
    p.ldx = d->ldx;
    p.x_bf16 = d->x_dtype == FP4_BF16;
    p.terms = d->terms;
    p.term_weights = d->term_weights;
    p.residual = d->residual;
    p.ldr = d->ldr;
    p.residual_out = d->residual_out;
    p.ldro = d->ldro;
    p.residual_bf16 = d->residual_dtype == FP4_BF16;
    p.gamma = d->gamma;
    p.gamma_bf16 = d->gamma_dtype == FP4_BF16;
    p.eps = d->eps;
    p.y = d->y;
    p.ldy = d->ldy;
    p.y_bf16 = d->y_dtype == FP4_BF16;
    return report_hip(launch_rmsnorm_quant(p, (hipStream_t)stream), "fp4_rmsnorm_quant");
}

fp4_status fp4_swiglu_quant(const fp4_swiglu8_desc* d, void* stream) {
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    fp4_status st = row_sizes(d->rows, d->cols);
    if (st) return st;
    if (d->reserved != 0) return report(FP4_ERR_INVALID_ARG, "reserved must be 0");
    if (!float_type(d->x_dtype)) return report(FP4_ERR_INVALID_ARG, "x_dtype must be FP4_F32 or FP4_BF16");
    if (d->rows == 0 || d->cols == 0) return report_ok();
    if (!d->x || !d->packed) return report(FP4_ERR_INVALID_ARG, "null pointer");
    SwigluParams p{};
    if ((st = code_output(d->rows, d->cols, d->grid, d->gran, d->tensor_scale, d->col_shift, d->packed, d->ldp, d->scales, &p.out))) return st;
    if ((st = matrix("x", d->x, d->rows, d->ldx, 2 * d->cols, d->x_dtype))) return st;
    p.rows = d->rows;
    p.cols = d->cols;
    p.x = d->x;
    p.ldx = d->ldx;
    p.x_bf16 = d->x_dtype == FP4_BF16;
    return report_hip(launch_swiglu_quant(p, (hipStream_t)stream), "fp4_swiglu_quant");
}

fp4_status fp4_quantize_block(const void* w, int32_t w_dtype, int64_t batch, int64_t n, int64_t k, int64_t ldw,
                              int64_t stride_w, fp4_grid grid, uint8_t* packed, int64_t ldp, int64_t stride_p,
                              float* scales, void* stream) {
    if (batch < 0 || n < 0 || k < 0) return report(FP4_ERR_INVALID_ARG, "bad sizes");
    if (!float_type(w_dtype)) return report(FP4_ERR_INVALID_ARG, "w_dtype must be FP4_F32 or FP4_BF16");
    if (k % 8 != 0) return report(FP4_ERR_UNSUPPORTED, "k must be a multiple of 8 (got %lld)", (long long)k);
    QGrid q;
    fp4_status st = fp8_grid(grid, &q);
    if (st) return st;
    if (batch == 0 || n == 0 || k == 0) return report_ok();
    if (!w || !packed || !scales) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if ((st = matrix("w", w, n, ldw, k, w_dtype))) return st;
    if (ldp < k || stride_w < 0 || stride_p < 0) return report(FP4_ERR_INVALID_ARG, "bad leading dimension or stride");
    if ((st = spans("packed", n, ldp)) || (st = spans("w", batch, stride_w)) || (st = spans("packed", batch, stride_p))) return st;
    if (!below(batch, blocks_of(n), 0x80000000ll) || !below(batch * blocks_of(n), blocks_of(k), 0x80000000ll))
        return report(FP4_ERR_UNSUPPORTED, "more than 2^31 scale blocks");
    if (overlap(batch, n, k, ldp, stride_p)) return report(FP4_ERR_INVALID_ARG, "the matrices of packed overlap");
    if (!aligned(packed, 8) || ldp % 8 != 0 || stride_p % 8 != 0 || (stride_w * size_of(w_dtype)) % 16 != 0 || !aligned(scales, 4))
        return report(FP4_ERR_ALIGNMENT, "packed, ldp and stride_p must be multiples of 8 bytes, stride_w of 16");
    BlockQuantParams p{};
    p.w = w;
    p.bf16 = w_dtype == FP4_BF16;
    p.batch = batch;
    p.n = n;
    p.k = k;
    p.ldw = ldw;
    p.stride_w = stride_w;
    p.e4m3 = q.e == 4;
    p.qmax = q.qmax;
    p.packed = packed;
    p.ldp = ldp;
    p.stride_p = stride_p;
    p.scales = scales;
    return report_hip(launch_quantize_block(p, (hipStream_t)stream), "fp4_quantize_block");
}

fp4_status fp4_gemm_block(const fp4_gemm_block_desc* d, void* stream) {
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    BlockGemmParams p{};
    fp4_status st = product_sizes(d->M, d->N, d->K);
    if (st) return st;
    if (d->reserved != 0) return report(FP4_ERR_INVALID_ARG, "reserved must be 0");
    if ((st = code_operand("a", d->a, d->lda, d->K, d->a_grid, &p.fa))) return st;
    if ((st = code_operand("w", d->w, d->ldw, d->K, d->w_grid, &p.fw))) return st;
    if ((st = product_output(d->y, d->M, d->ldy, d->N, d->y_dtype))) return st;
    if (d->lda_s < blocks_of(d->K) || d->ldw_s < blocks_of(d->K))
        return report(FP4_ERR_INVALID_ARG, "leading dimension of scales below ceil(K / 128)");
    if (d->lda_s > (1 << 20) || d->ldw_s > (1 << 20)) return report(FP4_ERR_UNSUPPORTED, "rows of scales must be shorter than 4 MiB");
    if (d->M == 0 || d->N == 0) return report_ok();
    if (!d->a || !d->a_scales || !d->w || !d->w_scales || !d->y) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (!aligned(d->a_scales, 4) || !aligned(d->w_scales, 4)) return report(FP4_ERR_ALIGNMENT, "scales must be 4-byte aligned");
    p.M = d->M;
    p.N = d->N;
    p.K = d->K;
    p.a = d->a;
    p.lda = d->lda;
    p.a_scales = d->a_scales;
    p.lda_s = d->lda_s;
    p.w = d->w;
    p.ldw = d->ldw;
    p.w_scales = d->w_scales;
    p.ldw_s = d->ldw_s;
    p.y = d->y;
    p.ldy = d->ldy;
    p.y_bf16 = d->y_dtype == FP4_BF16;
    p.slots_per_row = 1;
    return report_hip(launch_gemm_block(p, (hipStream_t)stream), "fp4_gemm_block");
}

size_t fp4_route_workspace_size(int64_t tokens, int32_t experts, int32_t top_k) {
    if (tokens <= 0 || experts < 1 || experts > 1024 || top_k < 1 || top_k > 32 || !below(tokens, top_k, 0x80000000ll)) return 0;
    return route_workspace_bytes(tokens, experts, top_k);
}

fp4_status fp4_route(const fp4_route_desc* d, void* workspace, size_t ws_bytes, void* stream) {
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    if (d->reserved != 0) return report(FP4_ERR_INVALID_ARG, "reserved must be 0");
    if (d->experts < 1 || d->experts > 1024) return report(FP4_ERR_UNSUPPORTED, "1 to 1024 experts (got %d)", d->experts);
    if (d->top_k < 1 || d->top_k > 32 || d->top_k > d->experts)
        return report(FP4_ERR_UNSUPPORTED, "top_k must be 1..32 and at most the experts (got %d)", d->top_k);
    if (d->tokens < 0 || !below(d->tokens, d->top_k, 0x80000000ll) || d->ld < d->experts)
        return report(FP4_ERR_INVALID_ARG, "bad sizes tokens=%lld ld=%lld", (long long)d->tokens, (long long)d->ld);
    fp4_status st = spans("logits", d->tokens, d->ld);
    if (st) return st;
    if (!float_type(d->logits_dtype)) return report(FP4_ERR_INVALID_ARG, "logits_dtype must be FP4_F32 or FP4_BF16");
    if (d->score != FP4_ROUTE_SOFTMAX && d->score != FP4_ROUTE_SIGMOID) return report(FP4_ERR_INVALID_ARG, "bad score %d", d->score);
    if (d->groups < 1 || d->groups > 64 || d->experts % d->groups != 0 || d->top_groups < 1 || d->top_groups > d->groups)
        return report(FP4_ERR_INVALID_ARG, "groups must be 1..64 and divide the experts, top_groups 1..groups");
    if (d->group_top != 1 && d->group_top != 2) return report(FP4_ERR_INVALID_ARG, "group_top must be 1 or 2");
    if (d->tokens != 0 && (d->offsets == nullptr) != (d->slots == nullptr)) return report(FP4_ERR_INVALID_ARG, "offsets and slots go together");
    if (!aligned(d->logits, size_of(d->logits_dtype)) || !aligned(d->bias, 4) || !aligned(d->experts_out, 4) ||
        !aligned(d->weights_out, 4) || !aligned(d->offsets, 4) || !aligned(d->slots, 4) || !aligned(workspace, 16))
        return report(FP4_ERR_ALIGNMENT, "pointers must be aligned to their types, the workspace to 16 bytes");
    if (d->tokens != 0 && (!d->logits || !d->experts_out || !d->weights_out)) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (d->tokens == 0 && !d->offsets) return report_ok();
    if (d->offsets) {
        const size_t need = fp4_route_workspace_size(d->tokens, d->experts, d->top_k);
        if (need && (!workspace || ws_bytes < need))
            return report(FP4_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? ws_bytes : (size_t)0);
    }
    RouteParams p{};
    p.tokens = d->tokens;
    p.experts = d->experts;
    p.top_k = d->top_k;
    p.logits = d->logits;
    p.ld = d->ld;
    p.logits_bf16 = d->logits_dtype == FP4_BF16;
    p.sigmoid = d->score == FP4_ROUTE_SIGMOID;
    p.bias = d->bias;
    p.groups = d->groups;
    p.top_groups = d->top_groups;
    p.group_top = d->group_top;
    p.renormalise = d->renormalise != 0;
    p.scale = d->scale;
    p.experts_out = d->experts_out;
    p.weights_out = d->weights_out;
    p.offsets = d->offsets;
    p.slots = d->slots;
    p.counts = (int32_t*)workspace;
    return report_hip(launch_route(p, (hipStream_t)stream), "fp4_route");
}

fp4_status fp4_gemm_experts(const fp4_gemm_experts_desc* d, void* stream) {
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    BlockGemmParams p{};
    fp4_status st = product_sizes(d->slots, d->N, d->K);
    if (st) return st;
    if (d->reserved != 0) return report(FP4_ERR_INVALID_ARG, "reserved must be 0");
    if (d->experts < 1 || d->experts > 1024) return report(FP4_ERR_UNSUPPORTED, "1 to 1024 experts (got %d)", d->experts);
    if (d->slots_per_row < 1) return report(FP4_ERR_INVALID_ARG, "slots_per_row must be positive");
    // the tiles of rows have to fit one launch (2^23 - 1 of 256 rows); every expert may have one
    // that is partly filled
    if (d->slots >= (1ll << 31) - (1 << 18)) return report(FP4_ERR_UNSUPPORTED, "slots must be below 2^31 - 2^18 (got %lld)", (long long)d->slots);
    if ((st = code_operand("a", d->a, d->lda, d->K, d->a_grid, &p.fa))) return st;
    if ((st = code_operand("w", d->w, d->ldw, d->K, d->w_grid, &p.fw))) return st;
    if ((st = product_output(d->y, d->slots, d->ldy, d->N, d->y_dtype))) return st;
    if (d->lda_s > (1 << 20)) return report(FP4_ERR_UNSUPPORTED, "rows of scales must be shorter than 4 MiB");
    if (d->lda_s < blocks_of(d->K)) return report(FP4_ERR_INVALID_ARG, "leading dimension of scales below ceil(K / 128)");
    if (d->stride_w < 0) return report(FP4_ERR_INVALID_ARG, "bad stride between experts");
    if (d->stride_w % 16 != 0) return report(FP4_ERR_ALIGNMENT, "experts must be a multiple of 16 bytes apart");
    if ((st = spans("w", d->experts, d->stride_w))) return st;
    if (d->slots == 0 || d->N == 0) return report_ok();
    if (!d->a || !d->a_scales || !d->w || !d->w_scales || !d->y || !d->offsets || !d->slot_list)
        return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (!aligned(d->a_scales, 4) || !aligned(d->w_scales, 4) || !aligned(d->offsets, 4) || !aligned(d->slot_list, 4))
        return report(FP4_ERR_ALIGNMENT, "scales, offsets and slots must be 4-byte aligned");
    const int64_t rows = (d->slots + d->slots_per_row - 1) / d->slots_per_row;
    if (!below(rows, d->lda, 0x7fff0000ll)) return report(FP4_ERR_UNSUPPORTED, "a must span less than 2 GiB");
    if (!below(rows, d->lda_s, 0x1fff0000ll)) return report(FP4_ERR_UNSUPPORTED, "a_scales must span less than 2 GiB");
    p.M = d->slots;
    p.N = d->N;
    p.K = d->K;
    p.a = d->a;
    p.lda = d->lda;
    p.a_scales = d->a_scales;
    p.lda_s = d->lda_s;
    p.w = d->w;
    p.ldw = d->ldw;
    p.stride_w = d->stride_w;
    p.w_scales = d->w_scales;
    p.ldw_s = blocks_of(d->K);
    p.stride_ws = blocks_of(d->N) * p.ldw_s;
    p.y = d->y;
    p.ldy = d->ldy;
    p.y_bf16 = d->y_dtype == FP4_BF16;
    p.experts = d->experts;
    p.slots_per_row = d->slots_per_row;
    p.offsets = d->offsets;
    p.slot_list = d->slot_list;
    return report_hip(launch_gemm_block(p, (hipStream_t)stream), "fp4_gemm_experts");
}

}  // extern "C"
