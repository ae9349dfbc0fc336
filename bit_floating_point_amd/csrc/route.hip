// Routing of tokens to experts, and the layout that the experts' products read.
//
// Choice: one wavefront per token, lane l holding experts l, 64 + l, ...; the scores are
// binary32, the top_k best are found one after another by a maximum over the wavefront.
// Layout: a stable counting sort of the tokens * top_k slots by expert -- counts per range
// of slots, then each range's slots placed behind those of the ranges before it -- so the
// order does not depend on timing.
#include "fp4_device.h"
#include "layer_internal.h"

namespace fp4 {

namespace {

constexpr int kRangeSlots = 2048;  // slots per workgroup of the layout
constexpr float kNone = -INFINITY;

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// lane and slot (i, with the expert i * 64 + lane) of the largest v, ties to the lowest
// expert; every lane returns the expert, or -1 if all are kNone
template <int EPL>
__device__ __forceinline__ int wave_argmax(const float (&v)[EPL], float* best) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < EPL; i++) m = fmaxf(m, v[i]);
    m = wave_max(m);
    *best = m;
    if (m == kNone) return -1;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const uint64_t b = __ballot(v[i] == m);
        if (b) return i * 64 + __ffsll((unsigned long long)b) - 1;
    }
    return -1;
}

}  // namespace

template <int EPL>
__global__ void __launch_bounds__(256) route_kernel(RouteParams p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 4 + wave;
    if (t >= p.tokens) return;
    float logit[EPL], score[EPL], key[EPL];
    float top = kNone;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = i * 64 + lane;
        float v = kNone;
        if (e < p.experts) {
            const int64_t at = t * p.ld + e;
            v = p.logits_bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p.logits)[at])
                              : reinterpret_cast<const float*>(p.logits)[at];
            if (!(fabsf(v) < INFINITY)) v = kNone;  // infinite or NaN: not usable
        }
        logit[i] = v;
        top = fmaxf(top, v);
    }
    float sum = 0.0f;
    if (!p.sigmoid) top = wave_max(top);
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const bool usable = logit[i] != kNone;
        score[i] = usable ? (p.sigmoid ? 1.0f / (1.0f + expf(-logit[i])) : expf(logit[i] - top)) : 0.0f;
        sum += score[i];
    }
    if (!p.sigmoid) sum = wave_add(sum);
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const bool usable = logit[i] != kNone;
        if (!p.sigmoid && usable) score[i] /= sum;
        const float b = usable && p.bias ? p.bias[i * 64 + lane] : 0.0f;
        key[i] = usable ? score[i] + b : kNone;
    }
    if (p.groups > 1) {
        const int size = p.experts / p.groups;
        // each group's value in lane g
        float value = kNone;
        for (int g = 0; g < p.groups; g++) {
            float k[EPL];
#pragma unroll
            for (int i = 0; i < EPL; i++) k[i] = (i * 64 + lane) / size == g ? key[i] : kNone;
            float a, b = kNone;
            const int first = wave_argmax<EPL>(k, &a);
            if (p.group_top == 2) {
#pragma unroll
                for (int i = 0; i < EPL; i++)
                    if (i * 64 + lane == first) k[i] = kNone;
                wave_argmax<EPL>(k, &b);
            }
            const float v = b == kNone ? a : a + b;
            if (lane == g) value = v;
        }
        uint64_t kept = 0;
        for (int j = 0; j < p.top_groups; j++) {
            float one[1] = {value}, best;
            const int g = wave_argmax<1>(one, &best);
            if (g < 0) break;
            kept |= 1ull << g;
            if (lane == g) value = kNone;
        }
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = i * 64 + lane;
            if (e < p.experts && !((kept >> (e / size)) & 1)) logit[i] = key[i] = kNone;
        }
    }
    if (!p.bias) {  // the logits have the scores' order, and neither round nor underflow
#pragma unroll
        for (int i = 0; i < EPL; i++) key[i] = logit[i];
    }
    // lane j ends up with the j-th choice
    int mine = -1;
    float weight = 0.0f;
    for (int j = 0; j < p.top_k; j++) {
        float best;
        const int e = wave_argmax<EPL>(key, &best);
        if (e < 0) break;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            if (i == e >> 6) s = score[i];
            if (i * 64 + lane == e) key[i] = kNone;
        }
        s = __shfl(s, e & 63, 64);
        if (lane == j) {
            mine = e;
            weight = s;
        }
    }
    if (p.renormalise) {
        const float total = wave_add(weight);
        weight = total > 0.0f ? weight / total : 0.0f;
    }
    if (lane < p.top_k) {
        p.experts_out[t * p.top_k + lane] = mine;
        p.weights_out[t * p.top_k + lane] = weight * p.scale;
    }
}

// counts[range][expert] (expert -1 last) of each range of slots
__global__ void __launch_bounds__(256) route_count_kernel(RouteParams p, int64_t nslots) {
    __shared__ int hist[1025];
    const int E = p.experts;
    for (int e = threadIdx.x; e <= E; e += 256) hist[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kRangeSlots;
    for (int i = threadIdx.x; i < kRangeSlots && first + i < nslots; i += 256) {
        const int e = p.experts_out[first + i];
        atomicAdd(&hist[e < 0 ? E : e], 1);  // counts: any order gives the same sum
    }
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += 256) p.counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// places each range's slots: behind all slots of lower experts and those of the same
// expert in earlier ranges
__global__ void __launch_bounds__(256) route_place_kernel(RouteParams p, int64_t nslots, int nranges) {
    __shared__ int before[1025];   // where this range's slots of an expert start
    __shared__ int total[1025];
    __shared__ int part[4][1025];  // per wavefront
    const int E = p.experts, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e <= E; e += 256) {
        int b = 0, all = 0;
        for (int r = 0; r < nranges; r++) {
            const int c = p.counts[(int64_t)r * (E + 1) + e];
            if (r < (int)blockIdx.x) b += c;
            all += c;
        }
        before[e] = b;
        total[e] = all;
        for (int w = 0; w < 4; w++) part[w][e] = 0;
    }
    __syncthreads();
    if (wave == 0) {  // exclusive sum of the totals over the experts
        int carry = 0;
        for (int e0 = 0; e0 <= E; e0 += 64) {
            const int e = e0 + lane;
            const int c = e <= E ? total[e] : 0;
            int s = c;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int u = __shfl_up(s, o, 64);
                if (lane >= o) s += u;
            }
            if (e <= E) {
                before[e] += carry + s - c;
                if (blockIdx.x == 0) p.offsets[e] = carry + s - c;
            }
            carry += __shfl(s, 63, 64);
        }
    }
    // wavefront w takes the w-th quarter of the range, 64 slots at a time
    constexpr int kQuarter = kRangeSlots / 4;
    const int64_t first = (int64_t)blockIdx.x * kRangeSlots + wave * kQuarter;
    for (int i = lane; i < kQuarter; i += 64)
        if (first + i < nslots) {
            const int e = p.experts_out[first + i];
            atomicAdd(&part[wave][e < 0 ? E : e], 1);
        }
    __syncthreads();
    for (int e = tid; e <= E; e += 256) {
        int b = before[e];
        for (int w = 0; w < 4; w++) {
            const int c = part[w][e];
            part[w][e] = b;
            b += c;
        }
    }
    __syncthreads();
    for (int i = 0; i < kQuarter; i += 64) {
        const int64_t s = first + i + lane;
        int e = -1;
        if (s < nslots) {
            e = p.experts_out[s];
            if (e < 0) e = E;
        }
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < 11; b++) {  // the lanes with this lane's expert
            const uint64_t ones = __ballot((e >> b) & 1);
            same &= ((e >> b) & 1) ? ones : ~ones;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int at = 0;
        if (e >= 0) at = part[wave][e];
        __builtin_amdgcn_wave_barrier();
        if (e >= 0) {
            p.slots[at + rank] = (int32_t)s;
            if (rank == 0) part[wave][e] = at + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// no tokens: all offsets 0
__global__ void route_empty_kernel(int32_t* offsets, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) offsets[i] = 0;
}

static int64_t route_ranges(int64_t tokens, int top_k) { return (tokens * top_k + kRangeSlots - 1) / kRangeSlots; }

size_t route_workspace_bytes(int64_t tokens, int32_t experts, int32_t top_k) {
    return (size_t)route_ranges(tokens, top_k) * (size_t)(experts + 1) * sizeof(int32_t);
}

hipError_t launch_route(const RouteParams& p, hipStream_t s) {
    if (p.tokens == 0) {
        route_empty_kernel<<<(p.experts + 256) / 256, 256, 0, s>>>(p.offsets, p.experts + 1);
        return hipGetLastError();
    }
    const dim3 grid((unsigned)((p.tokens + 3) / 4));
    if (p.experts <= 64) route_kernel<1><<<grid, 256, 0, s>>>(p);
    else if (p.experts <= 128) route_kernel<2><<<grid, 256, 0, s>>>(p);
    else if (p.experts <= 256) route_kernel<4><<<grid, 256, 0, s>>>(p);
    else if (p.experts <= 512) route_kernel<8><<<grid, 256, 0, s>>>(p);
    else route_kernel<16><<<grid, 256, 0, s>>>(p);
    if (p.offsets) {
        const int64_t nslots = p.tokens * p.top_k;
        const int64_t nranges = route_ranges(p.tokens, p.top_k);
        route_count_kernel<<<(unsigned)nranges, 256, 0, s>>>(p, nslots);
        route_place_kernel<<<(unsigned)nranges, 256, 0, s>>>(p, nslots, (int)nranges);
    }
    return hipGetLastError();
}

}  // namespace fp4
