/*
 * fp4_cache.h -- C ABI of libfp4, the paged key/value cache: rows of keys and values written
 * into pages as bf16 or as codes with scales, read back, and the attention of one new token per
 * sequence over them.
 *
 * The conventions of fp4.h hold (device pointers, caller-owned memory, asynchronous on
 * `stream`, no allocation, no synchronisation, host checks before any launch, thread safety,
 * status codes, fp4_last_error), with these additions:
 *   - Outputs may not overlap inputs.
 *   - What the host cannot see is safe whatever it holds: page numbers outside the cache,
 *     positions and lengths that are negative or past the page table, sequence numbers that are
 *     not there.  Each call says what they mean.
 *   - Work whose threads would pass 2^32, the most one launch takes, is split over launches.
 */
#ifndef FP4_CACHE_H_
#define FP4_CACHE_H_

#include "fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache: `pages` pages, each with page_size rows of head_dim keys and as many of values for
 * every kv head.  The row of slot j of kv head h in page p lies at
 *   k + p * stride_page + h * stride_head + j * stride_row   (bytes; v likewise),
 * so any order of pages, heads and slots is possible; rows may not overlap. */
typedef struct {
    void* k;
    void* v;
    int64_t pages;              /* 1 .. 2^31 - 1                                       */
    int64_t stride_page;        /* bytes, each a multiple of 16                        */
    int64_t stride_head;
    int64_t stride_row;         /* page_size * stride_row < 2^31                       */
    int32_t kv_heads;           /* 1 .. 65535                                          */
    int32_t page_size;          /* a power of two, 16 .. 65536                         */
    int32_t head_dim;           /* 64, 96, 128, 192 or 256                             */
    int32_t type;               /* FP4_BF16: rows of bf16; FP4_PACKED: codes of `grid` */
    fp4_grid grid;              /* E2M1 (two codes a byte), E4M3 or E5M2               */
    fp4_gran gran;              /* ROW: a scale per row; TENSOR: one f32 scale, given  */
    void* k_scales;             /* ROW: f32 or f16 [pages, kv_heads, page_size]        */
    void* v_scales;             /*   contiguous; TENSOR: f32, one value; else NULL     */
} fp4_kv_cache;

/* Rows of tokens.  Token i is position positions[i] of sequence sequence_of[i] (or of sequence i),
 * that is slot positions[i] % page_size of page
 *   page_table[sequence * ld_table + positions[i] / page_size].
 * A token has no row if its position is negative or past max_pages * page_size, its sequence
 * outside [0, sequences) or its page outside [0, pages). */
typedef struct {
    const int32_t* page_table;  /* int32 [sequences, max_pages], leading dim ld_table  */
    int64_t sequences;
    int64_t max_pages;          /* max_pages * page_size <= 2^30                       */
    int64_t ld_table;           /* elements; 0: all sequences have one row             */
    int64_t tokens;
    const int32_t* positions;   /* int32 [tokens]                                      */
    const int32_t* sequence_of; /* int32 [tokens], or NULL: token i is of sequence i   */
    void* k;                    /* [tokens, kv_heads * head_dim], leading dim ldk:     */
    int64_t ldk;                /*   inputs of a write, outputs of a read              */
    void* v;                    /* likewise, leading dim ldv                           */
    int64_t ldv;
    int32_t dtype;              /* of k and v: FP4_F32 or FP4_BF16                     */
    int32_t reserved;           /* must be 0                                           */
} fp4_cache_rows_desc;

/* ---- rows into the cache --------------------------------------------------------- */
/* The keys and values of the tokens into their rows.  Codes: per row s = fl32(amax / Qmax), no
 * less than 2^-126 unless amax is 0 (f16 scales: rounded to binary16, at most its largest
 * number), or the given s; codes of fl32(x * fl32(1/s)) as fp4_quantize_pack.  bf16: rounded to
 * nearest.  Tokens without a row are skipped; all other rows of the cache stay as they are.  No
 * two tokens of a call may have one row: what it holds then is a mixture of theirs.  Scales per row of
 * keys and of values may not share memory (one given scale may be both's). */
fp4_status fp4_cache_write(const fp4_kv_cache* cache, const fp4_cache_rows_desc* d, void* stream);

/* ---- rows out of the cache ------------------------------------------------------- */
/* The values that the tokens' rows hold (code value * scale, one rounding to binary32, one to
 * `dtype`) into k and v; zeros for tokens without a row. */
fp4_status fp4_cache_read(const fp4_kv_cache* cache, const fp4_cache_rows_desc* d, void* stream);

/* ---- attention of one new token per sequence -------------------------------------- */
typedef struct {
    int64_t sequences;
    int32_t heads;              /* query heads, a multiple of kv_heads: query head h reads
                                   kv head h / (heads / kv_heads)                      */
    int32_t q_dtype;            /* FP4_BF16 or FP4_F32                                 */
    const void* q;              /* [sequences, heads * head_dim], leading dim ldq      */
    int64_t ldq;
    const int32_t* page_table;  /* int32 [sequences, max_pages], leading dim ld_table  */
    int64_t max_pages;          /* max_pages * page_size <= 2^30                       */
    int64_t ld_table;
    const int32_t* lengths;     /* int32 [sequences]: positions, the new token's among them */
    int64_t max_length;         /* no length is larger (a larger one counts as this)   */
    int64_t window;             /* only the last `window` positions are seen; 0: all   */
    float scale;                /* factor of the products q k, |scale| < 2e38         */
    int32_t y_dtype;            /* FP4_BF16 or FP4_F32                                 */
    void* y;                    /* [sequences, heads * head_dim], leading dim ldy      */
    int64_t ldy;
    float* lse;                 /* f32 [sequences, heads], or NULL                     */
} fp4_attend_desc;

/* Workspace bytes that fp4_attend needs for these sizes (0: none). */
size_t fp4_attend_workspace_size(int64_t sequences, int32_t heads, int32_t kv_heads,
                                 int32_t head_dim, int64_t max_length, int64_t window);

/* For sequence b with n = min(lengths[b], max_length, max_pages * page_size) positions and each
 * query head, over the positions t that it sees -- max(0, n - window) <= t < n, their page in the
 * cache:
 *   z_t = scale * sum_d q_d K[t, d],  y = sum_t e^(z_t) V[t] / sum_t e^(z_t),
 *   lse = log sum_t e^(z_t);  a sequence that sees none has y = 0 and lse = -inf.
 * K and V are what the cache's rows stand for.  Rows that are not seen may hold anything.
 * Sums, maxima and exponentials are binary32.  On the matrix cores K, V and q are exact (an f32 q
 * as three bf16 terms) and the weights e^(z - m) are sums of two bf16 terms, three where q or y is
 * f32 (within 2^-18 and 2^-25 of themselves, as long as a weight times its row's scale is above
 * 2^-100).  Long sequences are split into parts that are joined in order: the result does not depend
 * on timing; which parts depends on the sizes and on the sequence's own length.
 * Binary32 must hold, over the positions that a sequence sees:
 *   |q_d K[t, d]| summed over d, K without its scale (|q_d| itself below 3.38e38);
 *   that times |scale| log2 e, and with a given scale of K times that too;
 *   z log2 e, which must stay below 1.5e38 in magnitude;
 *   2^8 |V[t, d]| summed over t, and 2^8 times a row's scale of V: weights pass 1 by as much between two
 *   moves of the running maximum, and the quotient is taken last.
 *   workspace  device scratch of at least fp4_attend_workspace_size() bytes, 16-byte aligned; what
 *              it holds before does not matter.  Calls that may overlap in time need one each  */
fp4_status fp4_attend(const fp4_kv_cache* cache, const fp4_attend_desc* d, void* workspace,
                      size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP4_CACHE_H_ */
