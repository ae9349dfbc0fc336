// Rows of keys and values into the pages of a cache, and out of them.
//
// One pass over HBM, which bounds both.  A row is D = 64 .. 256 values of one head: 8 values a lane
// (16 bytes of bf16), 8 .. 32 lanes a row, its largest magnitude a maximum over those lanes.  A
// lane takes the same 8 values of the key and of the value row, so that both loads are on
// their way before the row's place is known (three dependent loads: sequence, page, row).  A
// workgroup takes consecutive tokens of ONE head: their slots lie side by side in a page, and so
// do their scales (4 bytes a row, which would otherwise be one scattered write each).
//
// Measured (calls in a row): 16384 tokens of 40 heads of 128 from bf16 to E4M3 105 us, 4.8 TB/s of reads and writes, as a large
// copy; 12000 of them back 78 us, 4.8 TB/s; 4096 of 32 heads to E2M1 with f16 scales 21 us and back 16.  8 tokens of 8 heads: 3.6 us
// of kernel (three loads that wait for each other) of the call's 6.4.
#include "cache_internal.h"
#include "unit_codes.h"

namespace fp4 {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ RowPlace row_of(const CacheRowsParams& p, int64_t token) {
    return find_row(p.table, p.sequences, p.ld_table, p.capacity, p.c.page_log, p.c.pages, p.sequence_of ? p.sequence_of[token] : token,
                    p.positions[token]);
}

struct RowAt {
    int64_t row;    // byte offset of the row
    int64_t scale;  // index of its scale
};
__device__ __forceinline__ RowAt row_at(const CacheParams& c, RowPlace r, int head) {
    return RowAt{r.page * c.stride_page + head * c.stride_head + (int64_t)r.slot * c.stride_row,
                 (((int64_t)r.page * c.kv_heads + head) << c.page_log) + r.slot};
}

template <int STORE>
__device__ __forceinline__ void write_row8(const CacheParams& c, uint8_t* rows, void* scales, const RowAt& at, int col, int lanes,
                                           bool live, const float v[8]) {
    if constexpr (STORE == kStoreBf16) {
        if (live) put8(rows + at.row, true, col, v);
    } else {
        float s;
        if (c.scales == kScaleGiven) {
            s = *reinterpret_cast<const float*>(scales);
        } else {
            s = scale_of(lanes_max(amax8(v), lanes), c.qmax, c.rqmax);
            if (c.scales == kScaleRowF16) s = round_f16(fminf(s, 65504.0f));
            if (live && col == 0) {
                if (c.scales == kScaleRowF16) reinterpret_cast<__half*>(scales)[at.scale] = __float2half_rn(s);
                else reinterpret_cast<float*>(scales)[at.scale] = s;
            }
        }
        const float r = reciprocal(s);
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_amdgcn_fmed3f(v[i] * r, -c.qmax, c.qmax);
        if (!live) return;
        if constexpr (STORE == kStoreE2m1) {
            uint32_t w = 0;  // the convert that fp4_device.h's pack8 describes
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
            w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
            *reinterpret_cast<uint32_t*>(rows + at.row + col / 2) = w;
        } else {
            *reinterpret_cast<uint2*>(rows + at.row + col) = codes8<STORE == kStoreE4m3>(y);
        }
    }
}

// the raw codes (or bf16 values) of 8 columns
template <int STORE>
__device__ __forceinline__ uint4 load_row8(const uint8_t* rows, const RowAt& at, int col) {
    if constexpr (STORE == kStoreBf16) {
        return get16<true>(rows + at.row + 2 * col);
    } else if constexpr (STORE == kStoreE2m1) {
        return make_uint4(__builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(rows + at.row + col / 2)), 0, 0, 0);
    } else {
        const uint64_t u = __builtin_nontemporal_load(reinterpret_cast<const uint64_t*>(rows + at.row + col));
        return make_uint4((uint32_t)u, (uint32_t)(u >> 32), 0, 0);
    }
}
template <int STORE>
__device__ __forceinline__ void row8_values(const uint4& u, float s, float v[8]) {
    if constexpr (STORE == kStoreBf16) {
        raw8_to_float<true>(Raw8{u, u}, v);
        return;
    }
    auto put = [&](int i, auto pair) {
        v[i] = pair[0] * s;
        v[i + 1] = pair[1] * s;
    };
    if constexpr (STORE == kStoreE2m1) {
        put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.x, 1.0f, 0));
        put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.x, 1.0f, 1));
        put(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.x, 1.0f, 2));
        put(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(u.x, 1.0f, 3));
    } else if constexpr (STORE == kStoreE4m3) {
        put(0, __builtin_amdgcn_cvt_pk_f32_fp8((int)u.x, false));
        put(2, __builtin_amdgcn_cvt_pk_f32_fp8((int)u.x, true));
        put(4, __builtin_amdgcn_cvt_pk_f32_fp8((int)u.y, false));
        put(6, __builtin_amdgcn_cvt_pk_f32_fp8((int)u.y, true));
    } else if constexpr (STORE == kStoreE5m2) {
        put(0, __builtin_amdgcn_cvt_pk_f32_bf8((int)u.x, false));
        put(2, __builtin_amdgcn_cvt_pk_f32_bf8((int)u.x, true));
        put(4, __builtin_amdgcn_cvt_pk_f32_bf8((int)u.y, false));
        put(6, __builtin_amdgcn_cvt_pk_f32_bf8((int)u.y, true));
    }
}
__device__ __forceinline__ float load_scale(const CacheParams& c, const void* scales, int64_t at) {
    if (c.scales == kScaleRowF32) return reinterpret_cast<const float*>(scales)[at];
    if (c.scales == kScaleRowF16) return __half2float(reinterpret_cast<const __half*>(scales)[at]);
    return c.scales == kScaleGiven ? *reinterpret_cast<const float*>(scales) : 1.0f;
}

// workgroup (tokens, head), heads fastest: token and head of this lane's row, its columns
struct Unit {
    int64_t token;
    int head, col;
    bool live;
};
__device__ __forceinline__ Unit unit_of(const CacheRowsParams& p, int64_t first, int lane_log) {
    const uint32_t heads = (uint32_t)p.c.kv_heads, group = blockIdx.x / heads;
    Unit u;
    u.head = (int)(blockIdx.x - group * heads);
    u.token = first + (int64_t)group * (kThreads >> lane_log) + (threadIdx.x >> lane_log);
    u.col = (int)(threadIdx.x & ((1u << lane_log) - 1)) * 8;
    u.live = u.token < p.tokens && u.col < p.c.head_dim;
    return u;
}

}  // namespace

template <int STORE, bool BF16>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(CacheRowsParams p, int64_t first, int lane_log) {
    const Unit u = unit_of(p, first, lane_log);
    const int64_t at = (int64_t)u.head * p.c.head_dim + u.col;
    float k[8] = {}, v[8] = {};
    RowPlace place{-1, 0};
    if (u.live) {
        get8<true>(p.k_rows, BF16, u.token * p.ldk + at, k);
        get8<true>(p.v_rows, BF16, u.token * p.ldv + at, v);
        place = row_of(p, u.token);
    }
    const RowAt row = row_at(p.c, place, u.head);
    write_row8<STORE>(p.c, p.c.k, p.c.k_scales, row, u.col, 1 << lane_log, place.page >= 0, k);
    write_row8<STORE>(p.c, p.c.v, p.c.v_scales, row, u.col, 1 << lane_log, place.page >= 0, v);
}

template <int STORE, bool BF16>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(CacheRowsParams p, int64_t first, int lane_log) {
    const Unit u = unit_of(p, first, lane_log);
    if (!u.live) return;
    const int64_t at = (int64_t)u.head * p.c.head_dim + u.col;
    const RowPlace place = row_of(p, u.token);
    float k[8] = {}, v[8] = {};
    if (place.page >= 0) {
        const RowAt row = row_at(p.c, place, u.head);
        const uint4 kc = load_row8<STORE>(p.c.k, row, u.col), vc = load_row8<STORE>(p.c.v, row, u.col);
        const float ks = load_scale(p.c, p.c.k_scales, row.scale), vs = load_scale(p.c, p.c.v_scales, row.scale);
        row8_values<STORE>(kc, ks, k);
        row8_values<STORE>(vc, vs, v);
    }
    put8(p.k_rows, BF16, u.token * p.ldk + at, k);
    put8(p.v_rows, BF16, u.token * p.ldv + at, v);
}

namespace {

// `kernel` over all tokens, in launches of fewer than 2^32 threads
template <typename F>
hipError_t over_tokens(const CacheRowsParams& p, F kernel) {
    int lane_log = 3;
    while ((8 << lane_log) < p.c.head_dim) lane_log++;
    const int64_t rows = kThreads >> lane_log, most = max_workgroups(kThreads) / p.c.kv_heads * rows;
    for (int64_t first = 0; first < p.tokens; first += most) {
        const int64_t n = p.tokens - first < most ? p.tokens - first : most;
        kernel(dim3((unsigned)((n + rows - 1) / rows * p.c.kv_heads)), first, lane_log);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int STORE>
hipError_t write_rows(const CacheRowsParams& p, hipStream_t s) {
    return over_tokens(p, [&](dim3 grid, int64_t first, int lane_log) {
        if (p.bf16) cache_write_kernel<STORE, true><<<grid, kThreads, 0, s>>>(p, first, lane_log);
        else cache_write_kernel<STORE, false><<<grid, kThreads, 0, s>>>(p, first, lane_log);
    });
}
template <int STORE>
hipError_t read_rows(const CacheRowsParams& p, hipStream_t s) {
    return over_tokens(p, [&](dim3 grid, int64_t first, int lane_log) {
        if (p.bf16) cache_read_kernel<STORE, true><<<grid, kThreads, 0, s>>>(p, first, lane_log);
        else cache_read_kernel<STORE, false><<<grid, kThreads, 0, s>>>(p, first, lane_log);
    });
}

}  // namespace

hipError_t launch_cache_write(const CacheRowsParams& p, hipStream_t s) {
    switch (p.c.store) {
        case kStoreE4m3: return write_rows<kStoreE4m3>(p, s);
        case kStoreE5m2: return write_rows<kStoreE5m2>(p, s);
        case kStoreE2m1: return write_rows<kStoreE2m1>(p, s);
        default: return write_rows<kStoreBf16>(p, s);
    }
}
hipError_t launch_cache_read(const CacheRowsParams& p, hipStream_t s) {
    switch (p.c.store) {
        case kStoreE4m3: return read_rows<kStoreE4m3>(p, s);
        case kStoreE5m2: return read_rows<kStoreE5m2>(p, s);
        case kStoreE2m1: return read_rows<kStoreE2m1>(p, s);
        default: return read_rows<kStoreBf16>(p, s);
    }
}

}  // namespace fp4
