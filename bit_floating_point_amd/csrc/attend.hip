// Attention over a cache: the choice of a kernel (attend_kernel.h), and the join of a sequence's parts.
//
// Join: O = sum_i 2^(m_i - M) O_i, over sum_i 2^(m_i - M) l_i, in the order of the parts, one
// workgroup per sequence and query head.  Bound by reading the parts, which is little (4 bytes a
// value, parts of 256 positions or more): 4 to 5 us beside the parts' kernel, most of it launch and three
// loads that wait for each other.  Sequences of one part have their result already.
#include "attend_kernel.h"

namespace fp4 {

namespace {

constexpr int kJoinThreads = 256;
// Up to so many parts a head has a wavefront, else a workgroup (wavefront / workgroup, us of the whole call.  Two parts: 96 sequences of
// 1100, 64 heads, 50.6 / 55.9, 40 of 1500 35.9 / 37.5.  Four: 60 of 2100, 32 heads, 52.8 / 54.7, 40 of 2048, 64 heads, 38.0 / 39.4, but with
// few heads 4 of 1024 9.6 / 9.1 and 1 of 2000 11.7 / 11.2.  Eight: 4 of 4096 14.9 / 14.55.  Sixteen: 1 of 8192 14.5 / 13.3).
constexpr int kFewParts = 4;

__device__ __forceinline__ float block_reduce(float v, float* part, bool largest) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const float u = __shfl_xor(v, o, 64);
        v = largest ? fmaxf(v, u) : v + u;
    }
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < kJoinThreads / 64; i++) v = largest ? fmaxf(v, part[i]) : v + part[i];
    return v;
}

}  // namespace

// four columns of the result of head `unit`: O over the sum of weights
__device__ __forceinline__ void put_joined(const AttendParams& p, int64_t unit, int64_t sequence, int dim, int col, const float4& o, float top,
                                           float sum) {
    const float f = sum == 0.0f ? 0.0f : 1.0f / sum;
    attend::put4(p.y, p.y_bf16, sequence * p.ldy + (unit - sequence * p.heads) * dim + col, attend::f32x4{o.x * f, o.y * f, o.z * f, o.w * f});
    if (p.lse && col == 0) p.lse[unit] = attend::log_sum(top, sum);
}
__device__ __forceinline__ SplitRange range_of(const AttendParams& p, int64_t sequence) {
    return split_range(max(0, min(p.lengths[sequence], p.capacity)), p.window, p.split_log, p.least_log);
}
__device__ __forceinline__ void add4(float4& a, const float4& v, float w) {
    a.x = __builtin_fmaf(v.x, w, a.x), a.y = __builtin_fmaf(v.y, w, a.y);
    a.z = __builtin_fmaf(v.z, w, a.z), a.w = __builtin_fmaf(v.w, w, a.w);
}

// Many parts: a workgroup per head.  D columns as D / 4 lanes of four, the parts dealt to as many
// groups of lanes as there are.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(AttendParams p, int64_t first, int64_t) {
    constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
    __shared__ float weight[kMostSplits], part[2][kJoinThreads / 64];
    __shared__ float4 sums[kGroups][kLanes];
    const int64_t unit = first + blockIdx.x, sequence = unit / p.heads;
    const SplitRange range = range_of(p, sequence);
    const int used = range.used();
    if (used <= 1) return;
    const float* ml = p.part_ml + unit * p.splits * 2;
    const bool there = (int)threadIdx.x < used;
    const float m = there ? ml[2 * threadIdx.x] : attend::kNothing, l = there ? ml[2 * threadIdx.x + 1] : 0.0f;
    const float top = block_reduce(m, part[0], true);
    const float f = attend::power2(m - top);
    if (there) weight[threadIdx.x] = f;
    const float sum = block_reduce(f * l, part[1], false);  // its barrier orders the weights too
    const int col = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
    if (group < kGroups) {
        const float4* o = reinterpret_cast<const float4*>(p.part_o + unit * p.splits * D) + col;
        float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int i = group; i < used; i += kGroups) add4(a, o[(int64_t)i * kLanes], weight[i]);
        sums[group][col] = a;
    }
    __syncthreads();
    if (threadIdx.x < kLanes) {
        float4 o = sums[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < kGroups; i++) add4(o, sums[i][threadIdx.x], 1.0f);
        put_joined(p, unit, sequence, D, 4 * threadIdx.x, o, top, sum);
    }
}

// Few parts (at most 64): a wavefront per head, no barriers.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_few_kernel(AttendParams p, int64_t first, int64_t units) {
    constexpr int kLanes = D / 4, kGroups = 64 / kLanes;
    const int lane = threadIdx.x & 63;
    const int64_t unit = first + (int64_t)blockIdx.x * (kJoinThreads / 64) + (threadIdx.x >> 6), sequence = unit / p.heads;
    if (unit >= units) return;
    const SplitRange range = range_of(p, sequence);
    const int used = range.used();
    if (used <= 1) return;
    const float* ml = p.part_ml + unit * p.splits * 2;
    const bool there = lane < used;
    const float m = there ? ml[2 * lane] : attend::kNothing, l = there ? ml[2 * lane + 1] : 0.0f;
    const float top = wave_max(m), f = attend::power2(m - top);
    float sum = f * l;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) sum += __shfl_xor(sum, o, 64);
    const int col = lane % kLanes, group = lane / kLanes;
    const float4* o = reinterpret_cast<const float4*>(p.part_o + unit * p.splits * D) + col;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int from = 0; from < used; from += kGroups) {
        const int i = from + group;
        const float w = __shfl(f, i & 63, 64);
        if (group < kGroups && i < used) add4(a, o[(int64_t)i * kLanes], w);
    }
    float4 all = a;
#pragma unroll
    for (int i = 1; i < kGroups; i++) {
        all.x += __shfl(a.x, col + i * kLanes, 64), all.y += __shfl(a.y, col + i * kLanes, 64);
        all.z += __shfl(a.z, col + i * kLanes, 64), all.w += __shfl(a.w, col + i * kLanes, 64);
    }
    if (lane < kLanes) put_joined(p, unit, sequence, D, 4 * col, all, top, sum);
}

namespace {

template <int D>
hipError_t join(const AttendParams& p, hipStream_t s) {
    const int64_t units = p.sequences * p.heads;
    const bool few = p.splits <= kFewParts;
    const int64_t each = few ? kJoinThreads / 64 : 1, most = max_workgroups(kJoinThreads) * each;
    for (int64_t first = 0; first < units; first += most) {
        const int64_t n = units - first < most ? units - first : most;
        const dim3 grid((unsigned)((n + each - 1) / each));
        if (few) attend_join_few_kernel<D><<<grid, kJoinThreads, 0, s>>>(p, first, units);
        else attend_join_kernel<D><<<grid, kJoinThreads, 0, s>>>(p, first, units);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_attend(const AttendParams& p, hipStream_t s) {
    hipError_t e;
    switch (p.c.store) {
        case kStoreE4m3: e = launch_attend_e4m3(p, s); break;
        case kStoreE5m2: e = launch_attend_e5m2(p, s); break;
        case kStoreE2m1: e = launch_attend_e2m1(p, s); break;
        default: e = launch_attend_bf16(p, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    switch (p.c.head_dim) {
        case 64: return join<64>(p, s);
        case 96: return join<96>(p, s);
        case 128: return join<128>(p, s);
        case 192: return join<192>(p, s);
        default: return join<256>(p, s);
    }
}

}  // namespace fp4
