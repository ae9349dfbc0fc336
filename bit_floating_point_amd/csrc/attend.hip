// Attention over a cache: the choice of a kernel (attend_kernel.h), and the join of a sequence's parts.
//
// Join: O = sum_i 2^(m_i - M) O_i, over sum_i 2^(m_i - M) l_i, in the order of the parts, one
// workgroup per sequence and query head.  Bound by reading the parts, which is little (4 bytes a
// value, parts of 512 positions or more).  Sequences of one part have their result already.
#include "attend_kernel.h"

namespace fp4 {

namespace {

constexpr int kJoinThreads = 256;

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

// D columns as D / 4 lanes of four, the parts dealt to as many groups of lanes as there are
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(AttendParams p, int64_t first) {
    constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
    __shared__ float weight[kMostSplits], part[2][kJoinThreads / 64];
    __shared__ float4 sums[kGroups][kLanes];
    const int64_t unit = first + blockIdx.x, sequence = unit / p.heads;
    const int32_t length = max(0, min(p.lengths[sequence], p.capacity));
    const SplitRange range = split_range(length, p.window, p.splits);
    if (range.used <= 1) return;
    const float* ml = p.part_ml + unit * p.splits * 2;
    const bool there = (int)threadIdx.x < range.used;
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
        for (int i = group; i < range.used; i += kGroups) {
            const float4 v = o[(int64_t)i * kLanes];
            const float w = weight[i];
            a.x = __builtin_fmaf(v.x, w, a.x), a.y = __builtin_fmaf(v.y, w, a.y);
            a.z = __builtin_fmaf(v.z, w, a.z), a.w = __builtin_fmaf(v.w, w, a.w);
        }
        sums[group][col] = a;
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float o = 0.0f;
#pragma unroll
        for (int i = 0; i < kGroups; i++) o += reinterpret_cast<const float*>(&sums[i][0])[threadIdx.x];
        const float y = sum > 0.0f ? o / sum : sum == 0.0f ? 0.0f : sum;
        const int64_t to = sequence * p.ldy + (unit - sequence * p.heads) * D + threadIdx.x;
        if (p.y_bf16) reinterpret_cast<__bf16*>(p.y)[to] = (__bf16)y;
        else reinterpret_cast<float*>(p.y)[to] = y;
        if (p.lse && threadIdx.x == 0) p.lse[unit] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0x1.62e43p-1f;
    }
}

hipError_t launch_attend(const AttendParams& p, hipStream_t s) {
    hipError_t e;
    switch (p.c.store) {
        case kStoreE4m3: e = launch_attend_e4m3(p, s); break;
        case kStoreE5m2: e = launch_attend_e5m2(p, s); break;
        case kStoreE2m1: e = launch_attend_e2m1(p, s); break;
        default: e = launch_attend_bf16(p, s); break;
    }
    if (e != hipSuccess || p.splits == 1) return e;
    const int64_t units = p.sequences * p.heads, most = max_workgroups(kJoinThreads);
    for (int64_t first = 0; first < units; first += most) {
        const dim3 grid((unsigned)(units - first < most ? units - first : most));
        switch (p.c.head_dim) {
            case 64: attend_join_kernel<64><<<grid, kJoinThreads, 0, s>>>(p, first); break;
            case 96: attend_join_kernel<96><<<grid, kJoinThreads, 0, s>>>(p, first); break;
            case 128: attend_join_kernel<128><<<grid, kJoinThreads, 0, s>>>(p, first); break;
            case 192: attend_join_kernel<192><<<grid, kJoinThreads, 0, s>>>(p, first); break;
            default: attend_join_kernel<256><<<grid, kJoinThreads, 0, s>>>(p, first); break;
        }
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fp4
