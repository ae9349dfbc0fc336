// Internal declarations of the key/value cache (include/fp4_cache.h): parameters that the
// host layer (cache_api.cpp) passes to the HIP kernels, and the rule that splits a sequence.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attend_split.h"
#include "layer_internal.h"

namespace fp4 {

// what a cache's rows hold
enum CacheStore : int32_t { kStoreBf16 = 0, kStoreE4m3 = 1, kStoreE5m2 = 2, kStoreE2m1 = 3 };
// scales: none (bf16), one f32 given, one f32 or f16 a row
enum CacheScales : int32_t { kScaleNone = 0, kScaleGiven = 1, kScaleRowF32 = 2, kScaleRowF16 = 3 };

struct CacheParams {
    uint8_t* k;
    uint8_t* v;
    int64_t stride_page, stride_head;  // bytes
    uint32_t stride_row;
    int32_t pages, kv_heads, page_log, head_dim;
    int32_t store;   // CacheStore
    int32_t scales;  // CacheScales
    float qmax, rqmax;
    void* k_scales;
    void* v_scales;
};

// rows of tokens: in (write) or out (read)
struct CacheRowsParams {
    CacheParams c;
    const int32_t* table;
    int64_t sequences, ld_table;
    int32_t capacity;  // positions of the page table
    const int32_t* positions;
    const int32_t* sequence_of;
    int64_t tokens;
    void* k_rows;
    void* v_rows;
    int64_t ldk, ldv;  // elements
    int32_t bf16;
};
hipError_t launch_cache_write(const CacheRowsParams& p, hipStream_t s);
hipError_t launch_cache_read(const CacheRowsParams& p, hipStream_t s);

struct AttendParams {
    CacheParams c;
    int64_t sequences;
    int32_t heads, share;  // query heads; of one kv head
    const void* q;
    int64_t ldq;
    int32_t q_bf16, y_bf16;
    const int32_t* table;
    int64_t ld_table;
    int32_t capacity;  // positions a sequence can have
    int32_t window;    // 0: none
    const int32_t* lengths;
    float scale_log2;  // scale * log2 e: exponentials are powers of two
    void* y;
    int64_t ldy;
    float* lse;
    int32_t splits;    // parts of a sequence, at most: a power of two
    int32_t split_log;
    PartRule least_log;  // how short parts may be
    float* part_o;     // [sequences, heads, splits, head_dim], workspace
    float* part_ml;    // [sequences, heads, splits, 2]: maximum, sum
};
hipError_t launch_attend(const AttendParams& p, hipStream_t s);

}  // namespace fp4
