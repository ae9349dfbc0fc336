// Host layer of the key/value cache (include/fp4_cache.h): argument validation (before any
// launch) and dispatch to the HIP kernels.
#include "../../include/fp4_cache.h"
#include "cache_internal.h"

using namespace fp4;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool float_type(int32_t t) { return t == FP4_F32 || t == FP4_BF16; }

int64_t size_of(int32_t t) { return t == FP4_BF16 ? 2 : 4; }

// a * b stays below `limit` (a, b >= 0)
bool below(int64_t a, int64_t b, int64_t limit) { return b == 0 || a <= (limit - 1) / b; }

constexpr int64_t kMostPositions = 1ll << 30;  // of a sequence
constexpr int64_t kMostHeads = 65536;

// the matrix [rows, cols] at p: leading dimension and alignment of 16-byte accesses
fp4_status matrix(const char* name, const void* p, int64_t rows, int64_t ld, int64_t cols, int32_t type) {
    if (ld < cols) return report(FP4_ERR_INVALID_ARG, "leading dimension of %s below its columns", name);
    if (!below(rows, ld, 1ll << 60)) return report(FP4_ERR_UNSUPPORTED, "%s spans more than 2^60 elements", name);
    if (!aligned(p, 16) || ld % (16 / size_of(type)) != 0)
        return report(FP4_ERR_ALIGNMENT, "%s must be 16-byte aligned, its rows a multiple of 16 bytes apart", name);
    return FP4_OK;
}

// Rows of `bytes` bytes in three dimensions: whether each dimension's stride clears what the
// smaller ones span, so that no two rows share a byte and every offset has 62 bits.
fp4_status row_layout(const fp4_kv_cache& c, int64_t bytes) {
    struct { int64_t stride, count; } d[3] = {{c.stride_row, c.page_size}, {c.stride_head, c.kv_heads}, {c.stride_page, c.pages}};
    for (int i = 0; i < 3; i++)  // in the order of their strides
        for (int j = i + 1; j < 3; j++)
            if (d[j].stride < d[i].stride) {
                const auto t = d[i];
                d[i] = d[j];
                d[j] = t;
            }
    int64_t span = bytes;
    for (const auto& e : d) {
        if (e.count == 1) continue;
        if (e.stride < span) return report(FP4_ERR_INVALID_ARG, "rows of the cache overlap");
        if (!below(e.count, e.stride, 1ll << 61)) return report(FP4_ERR_UNSUPPORTED, "the cache spans more than 2^61 bytes");
        span += (e.count - 1) * e.stride;
    }
    return FP4_OK;
}

fp4_status cache_of(const fp4_kv_cache* cache, CacheParams* out) {
    if (!cache) return report(FP4_ERR_INVALID_ARG, "null cache");
    const fp4_kv_cache& c = *cache;
    if (c.pages < 1 || c.pages > 0x7fffffff || c.kv_heads < 1 || c.kv_heads > 65535)
        return report(FP4_ERR_INVALID_ARG, "bad sizes pages=%lld kv_heads=%d", (long long)c.pages, c.kv_heads);
    if (c.page_size < 16 || c.page_size > 65536 || (c.page_size & (c.page_size - 1)))
        return report(FP4_ERR_UNSUPPORTED, "page_size must be a power of two in [16, 65536] (got %d)", c.page_size);
    if (c.head_dim != 64 && c.head_dim != 96 && c.head_dim != 128 && c.head_dim != 192 && c.head_dim != 256)
        return report(FP4_ERR_UNSUPPORTED, "head_dim must be 64, 96, 128, 192 or 256 (got %d)", c.head_dim);
    int64_t bytes;
    if (c.type == FP4_BF16) {
        if (c.k_scales || c.v_scales) return report(FP4_ERR_INVALID_ARG, "a bf16 cache has no scales");
        out->store = kStoreBf16;
        out->scales = kScaleNone;
        bytes = 2 * c.head_dim;
    } else if (c.type == FP4_PACKED) {
        QGrid q;
        fp4_status st = grid_table(c.grid, &q);
        if (st) return st;
        if (q.kind != 0 || !(q.is_e2m1 || q.bits == 8)) return report(FP4_ERR_UNSUPPORTED, "the grid must be E2M1, E4M3 or E5M2");
        if (c.gran.reserved != 0) return report(FP4_ERR_INVALID_ARG, "fp4_gran.reserved must be 0");
        if (c.gran.mode != FP4_SCALE_ROW && c.gran.mode != FP4_SCALE_TENSOR)
            return report(c.gran.mode == FP4_SCALE_GROUP ? FP4_ERR_UNSUPPORTED : FP4_ERR_INVALID_ARG, "the scales of a cache are per ROW or TENSOR");
        if (c.gran.scale_dtype != FP4_F32 && c.gran.scale_dtype != FP4_F16)
            return report(FP4_ERR_INVALID_ARG, "scale dtype must be FP4_F32 or FP4_F16");
        if (c.gran.mode == FP4_SCALE_TENSOR && c.gran.scale_dtype != FP4_F32) return report(FP4_ERR_UNSUPPORTED, "per-tensor scales are f32 only");
        if (!c.k_scales || !c.v_scales) return report(FP4_ERR_INVALID_ARG, "a cache of codes needs k_scales and v_scales");
        out->store = q.is_e2m1 ? kStoreE2m1 : q.e == 4 ? kStoreE4m3 : kStoreE5m2;
        out->scales = c.gran.mode == FP4_SCALE_TENSOR ? kScaleGiven : c.gran.scale_dtype == FP4_F16 ? kScaleRowF16 : kScaleRowF32;
        out->qmax = q.qmax;
        out->rqmax = 1.0f / q.qmax;
        bytes = c.head_dim * (q.is_e2m1 ? 4 : 8) / 8;
    } else {
        return report(FP4_ERR_INVALID_ARG, "the type of a cache must be FP4_BF16 or FP4_PACKED (got %d)", c.type);
    }
    if (c.stride_page < 0 || c.stride_head < 0 || c.stride_row < 0) return report(FP4_ERR_INVALID_ARG, "negative stride");
    fp4_status st = row_layout(c, bytes);
    if (st) return st;
    if (!below(c.page_size, c.stride_row, 1ll << 31)) return report(FP4_ERR_UNSUPPORTED, "the rows of a head's page must span less than 2 GiB");
    if (!c.k || !c.v) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (c.k == c.v) return report(FP4_ERR_INVALID_ARG, "k and v are the same rows");
    if (!aligned(c.k, 16) || !aligned(c.v, 16) || c.stride_page % 16 != 0 || c.stride_head % 16 != 0 || c.stride_row % 16 != 0 ||
        !aligned(c.k_scales, 16) || !aligned(c.v_scales, 16))
        return report(FP4_ERR_ALIGNMENT, "the cache's pointers and strides must be multiples of 16 bytes");
    out->k = (uint8_t*)c.k;
    out->v = (uint8_t*)c.v;
    out->stride_page = c.stride_page;
    out->stride_head = c.stride_head;
    out->stride_row = (uint32_t)c.stride_row;
    out->pages = (int32_t)c.pages;
    out->kv_heads = c.kv_heads;
    out->page_log = __builtin_ctz((unsigned)c.page_size);
    out->head_dim = c.head_dim;
    out->k_scales = c.k_scales;
    out->v_scales = c.v_scales;
    return FP4_OK;
}

// Scales of rows that a write stores: keys' and values' share no memory.  (Rows span less than 2^61 bytes, 32 or more each.)
fp4_status scales_apart(const CacheParams& c) {
    if (c.scales != kScaleRowF32 && c.scales != kScaleRowF16) return FP4_OK;
    const uint64_t bytes = (((uint64_t)c.pages * (uint64_t)c.kv_heads) << c.page_log) * (c.scales == kScaleRowF16 ? 2 : 4);
    const uintptr_t k = reinterpret_cast<uintptr_t>(c.k_scales), v = reinterpret_cast<uintptr_t>(c.v_scales);
    return (k < v ? v - k : k - v) < bytes ? report(FP4_ERR_INVALID_ARG, "k_scales and v_scales share memory") : FP4_OK;
}

// the page table's sizes; *capacity: positions that a sequence can have
fp4_status table_of(const int32_t* table, int64_t sequences, int64_t max_pages, int64_t ld, const CacheParams& c, int32_t* capacity) {
    if (sequences < 0 || sequences > 0x7fffffff || max_pages < 0)
        return report(FP4_ERR_INVALID_ARG, "bad sizes sequences=%lld max_pages=%lld", (long long)sequences, (long long)max_pages);
    if (!below(max_pages, 1ll << c.page_log, kMostPositions + 1)) return report(FP4_ERR_UNSUPPORTED, "a sequence has at most 2^30 positions");
    if (ld != 0 && ld < max_pages) return report(FP4_ERR_INVALID_ARG, "ld_table neither 0 nor at least max_pages");
    if (!below(sequences, ld, 1ll << 60)) return report(FP4_ERR_UNSUPPORTED, "page_table spans more than 2^60 elements");
    if (!table && sequences > 0 && max_pages > 0) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (!aligned(table, 4)) return report(FP4_ERR_ALIGNMENT, "page_table must be 4-byte aligned");
    *capacity = (int32_t)(max_pages << c.page_log);
    return FP4_OK;
}

// what a call on rows of tokens launches with
fp4_status rows_of(const fp4_kv_cache* cache, const fp4_cache_rows_desc* d, CacheRowsParams* p) {
    fp4_status st = cache_of(cache, &p->c);
    if (st) return st;
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    if (d->reserved != 0) return report(FP4_ERR_INVALID_ARG, "reserved must be 0");
    if (d->tokens < 0) return report(FP4_ERR_INVALID_ARG, "bad sizes tokens=%lld", (long long)d->tokens);
    if (!float_type(d->dtype)) return report(FP4_ERR_INVALID_ARG, "dtype must be FP4_F32 or FP4_BF16");
    if ((st = table_of(d->page_table, d->sequences, d->max_pages, d->ld_table, p->c, &p->capacity))) return st;
    const int64_t cols = (int64_t)p->c.kv_heads * p->c.head_dim;
    if ((st = matrix("k", d->k, d->tokens, d->ldk, cols, d->dtype)) || (st = matrix("v", d->v, d->tokens, d->ldv, cols, d->dtype))) return st;
    if (d->tokens > 0 && (!d->k || !d->v || !d->positions)) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (!aligned(d->positions, 4) || !aligned(d->sequence_of, 4))
        return report(FP4_ERR_ALIGNMENT, "positions and sequence_of must be 4-byte aligned");
    p->table = d->page_table;
    p->sequences = d->sequences;
    p->ld_table = d->ld_table;
    p->positions = d->positions;
    p->sequence_of = d->sequence_of;
    p->tokens = d->tokens;
    p->k_rows = d->k;
    p->v_rows = d->v;
    p->ldk = d->ldk;
    p->ldv = d->ldv;
    p->bf16 = d->dtype == FP4_BF16;
    return FP4_OK;
}

// sizes of an attention call that its workspace goes by
bool attend_sizes(int64_t sequences, int32_t heads, int32_t kv_heads, int64_t max_length, int64_t window) {
    return sequences > 0 && sequences <= 0x7fffffff && kv_heads >= 1 && kv_heads <= 65535 && heads >= 1 && heads <= kMostHeads &&
           heads % kv_heads == 0 && max_length > 0 && window >= 0;
}
int64_t capped(int64_t length) { return length < kMostPositions ? length : kMostPositions; }

}  // namespace

extern "C" {

fp4_status fp4_cache_write(const fp4_kv_cache* cache, const fp4_cache_rows_desc* d, void* stream) {
    CacheRowsParams p{};
    fp4_status st = rows_of(cache, d, &p);
    if (st) return st;
    if (p.tokens == 0 || p.sequences == 0 || p.capacity == 0) return report_ok();  // no token has a row
    if ((st = scales_apart(p.c))) return st;
    return report_hip(launch_cache_write(p, (hipStream_t)stream), "fp4_cache_write");
}

fp4_status fp4_cache_read(const fp4_kv_cache* cache, const fp4_cache_rows_desc* d, void* stream) {
    CacheRowsParams p{};
    const fp4_status st = rows_of(cache, d, &p);
    if (st) return st;
    if (p.tokens == 0) return report_ok();
    if (p.k_rows == p.v_rows) return report(FP4_ERR_INVALID_ARG, "k and v are the same rows");
    return report_hip(launch_cache_read(p, (hipStream_t)stream), "fp4_cache_read");
}

size_t fp4_attend_workspace_size(int64_t sequences, int32_t heads, int32_t kv_heads, int32_t head_dim, int64_t max_length, int64_t window) {
    if (!attend_sizes(sequences, heads, kv_heads, max_length, window) || head_dim < 1 || head_dim > 256) return 0;
    const int64_t splits = split_count(sequences, heads, kv_heads, capped(max_length), window);
    return splits == 1 ? 0 : (size_t)(sequences * heads * splits * (head_dim + 2)) * sizeof(float);
}

fp4_status fp4_attend(const fp4_kv_cache* cache, const fp4_attend_desc* d, void* workspace, size_t ws_bytes, void* stream) {
    AttendParams p{};
    fp4_status st = cache_of(cache, &p.c);
    if (st) return st;
    if (!d) return report(FP4_ERR_INVALID_ARG, "null descriptor");
    if (!float_type(d->q_dtype) || !float_type(d->y_dtype)) return report(FP4_ERR_INVALID_ARG, "q_dtype and y_dtype must be FP4_F32 or FP4_BF16");
    if (d->heads < 1 || d->heads % p.c.kv_heads != 0) return report(FP4_ERR_INVALID_ARG, "heads must be a multiple of kv_heads (got %d)", d->heads);
    if (d->heads > kMostHeads) return report(FP4_ERR_UNSUPPORTED, "at most 65536 heads (got %d)", d->heads);
    if (d->max_length < 0 || d->window < 0) return report(FP4_ERR_INVALID_ARG, "max_length and window must not be negative");
    if (!(d->scale > -2.0e38f && d->scale < 2.0e38f)) return report(FP4_ERR_INVALID_ARG, "scale must be below 2e38");
    if ((st = table_of(d->page_table, d->sequences, d->max_pages, d->ld_table, p.c, &p.capacity))) return st;
    const int64_t cols = (int64_t)d->heads * p.c.head_dim;
    if ((st = matrix("q", d->q, d->sequences, d->ldq, cols, d->q_dtype)) || (st = matrix("y", d->y, d->sequences, d->ldy, cols, d->y_dtype))) return st;
    if (d->sequences == 0) return report_ok();
    if (!d->q || !d->y || !d->lengths) return report(FP4_ERR_INVALID_ARG, "null pointer");
    if (!aligned(d->lengths, 4) || !aligned(d->lse, 4) || !aligned(workspace, 16))
        return report(FP4_ERR_ALIGNMENT, "lengths and lse must be 4-byte aligned, the workspace 16-byte");
    if (d->max_length < p.capacity) p.capacity = (int32_t)d->max_length;
    p.window = d->window < kMostPositions ? (int32_t)d->window : 0;
    p.splits = p.capacity ? split_count(d->sequences, d->heads, p.c.kv_heads, p.capacity, p.window) : 1;
    p.split_log = __builtin_ctz((unsigned)p.splits);
    p.least_log = part_least_log(attend_units(d->sequences, d->heads, p.c.kv_heads));
    const int64_t values = d->sequences * d->heads * p.splits;
    if (p.splits > 1) {
        const size_t need = (size_t)(values * (p.c.head_dim + 2)) * sizeof(float);
        if (!workspace || ws_bytes < need) return report(FP4_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace ? ws_bytes : (size_t)0);
        p.part_o = (float*)workspace;
        p.part_ml = p.part_o + values * p.c.head_dim;
    }
    p.sequences = d->sequences;
    p.heads = d->heads;
    p.share = d->heads / p.c.kv_heads;
    p.q = d->q;
    p.ldq = d->ldq;
    p.q_bf16 = d->q_dtype == FP4_BF16;
    p.y_bf16 = d->y_dtype == FP4_BF16;
    p.table = d->page_table;
    p.ld_table = d->ld_table;
    p.lengths = d->lengths;
    p.scale_log2 = d->scale * 0x1.715476p+0f;
    p.y = d->y;
    p.ldy = d->ldy;
    p.lse = d->lse;
    return report_hip(launch_attend(p, (hipStream_t)stream), "fp4_attend");
}

}  // extern "C"
