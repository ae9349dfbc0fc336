// Routing of tokens to experts, and the layout that the experts' products read.
//
// Choice: one wavefront per token.  A group of experts takes LG lanes (a power of two, all 64
// without groups), each lane EPL consecutive experts: the order of (lane, place) is the order
// of the experts, which is how ties go to the lower one.  A lane sorts its keys once; then the
// best of all lanes' heads is taken top_k times, its lane moving on to the next of its list.
// Groups are compared by merging the lanes' two best.  Scores, sums and keys are binary32.
//
// Layout: a stable counting sort of the tokens * top_k slots by expert.  The choice leaves the
// counts of at most 256 ranges of tokens; every workgroup that places slots adds up the ranges
// before its own.  The order does not depend on timing.  Few tokens: one workgroup does all.
//
// Bound by the vector instructions of the selection.
#include "fp4_device.h"
#include "layer_internal.h"

namespace fp4 {

namespace {

constexpr float kNone = -INFINITY;  // key of an expert that cannot be chosen
constexpr int kMaxE = 1024;
constexpr int kRanges = 256;        // ranges of tokens counted apart, at most
constexpr int kSmallSlots = 1024, kSmallTokens = 64;  // one workgroup routes and places these
constexpr float kLog2e = 0x1.715476p+0f;

// v of the lane that a DPP control names (lanes without a source keep v)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), CTRL, 0xF, 0xF, false));
}

// largest v of the wavefront, uniform
__device__ __forceinline__ float max64(float v) {
    v = fmaxf(v, dpp<0xB1>(v));   // neighbours
    v = fmaxf(v, dpp<0x4E>(v));   // pairs
    v = fmaxf(v, dpp<0x141>(v));  // halves of 8
    v = fmaxf(v, dpp<0x140>(v));  // halves of 16
    v = fmaxf(v, dpp<0x142>(v));  // row 0 into 1, 2 into 3
    v = fmaxf(v, dpp<0x143>(v));  // rows 0, 1 into 2, 3
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

__device__ __forceinline__ float sum64(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// score of a usable logit; softmax: top is the largest logit, rsum one over the sum
__device__ __forceinline__ float score_of(float l, bool sigmoid, float top, float rsum) {
    if (sigmoid) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * l));
    return __builtin_amdgcn_exp2f(kLog2e * (l - top)) * rsum;
}

__device__ __forceinline__ float logit_at(const RouteParams& p, int64_t t, int e) {
    const int64_t at = t * p.ld + e;
    return p.logits_bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p.logits)[at])
                         : reinterpret_cast<const float*>(p.logits)[at];
}

// The choice for token t, written out; lane j < top_k returns the j-th expert (or -1).
template <int EPL>
__device__ __forceinline__ int choose(const RouteParams& p, int64_t t, int lane, int lg_bits, const float* bias) {
    const int group = lane >> lg_bits, size = p.experts / p.groups;
    const int place = (lane & ((1 << lg_bits) - 1)) * EPL;  // within the group
    const int base = group * size + place, count = group < p.groups ? min(size - place, EPL) : 0;
    float key[EPL];
    int idx[EPL];
    float top = kNone;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        float v = kNone;
        if (i < count) {
            v = logit_at(p, t, base + i);
            if (!(fabsf(v) < INFINITY)) v = kNone;  // infinite or NaN: not usable
        }
        key[i] = v;
        idx[i] = base + i;
        top = fmaxf(top, v);
    }
    float rsum = 0.0f;
    if (!p.sigmoid) {
        top = max64(top);
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) s += key[i] == kNone ? 0.0f : __builtin_amdgcn_exp2f(kLog2e * (key[i] - top));
        rsum = 1.0f / sum64(s);
    }
    // Keys: score + bias; without a bias the logit, which has the scores' order and neither
    // rounds nor underflows.
    if (bias) {
#pragma unroll
        for (int i = 0; i < EPL; i++)
            if (key[i] != kNone) key[i] = score_of(key[i], p.sigmoid, top, rsum) + bias[base + i];
    }
#pragma unroll
    for (int a = 0; a + 1 < EPL; a++) {  // largest first; equal keys stay in order
#pragma unroll
        for (int b = EPL - 1; b > a; b--) {
            const bool swap = key[b] > key[b - 1];
            const float k = key[b];
            const int x = idx[b];
            key[b] = swap ? key[b - 1] : k;
            idx[b] = swap ? idx[b - 1] : x;
            key[b - 1] = swap ? k : key[b - 1];
            idx[b - 1] = swap ? x : idx[b - 1];
        }
    }
    if (p.groups > 1) {
        // the group's two best values, in all of its lanes
        float a = key[0], b = EPL > 1 ? key[EPL > 1 ? 1 : 0] : kNone;
        if (!bias) {
            a = a == kNone ? a : score_of(a, p.sigmoid, top, rsum);
            b = b == kNone ? b : score_of(b, p.sigmoid, top, rsum);
        }
        for (int o = 1; o < (1 << lg_bits); o <<= 1) {
            const float c = __shfl_xor(a, o, 64), d = __shfl_xor(b, o, 64);
            b = fmaxf(fminf(a, c), fmaxf(b, d));
            a = fmaxf(a, c);
        }
        float value = p.group_top == 2 && b != kNone ? a + b : a;
        if (place != 0 || group >= p.groups) value = kNone;
        uint64_t kept = 0;
        for (int j = 0; j < p.top_groups; j++) {
            const float m = max64(value);
            const uint64_t at = __ballot(value == m && m != kNone);
            if (!at) break;
            const int l = __ffsll((unsigned long long)at) - 1;
            kept |= 1ull << (l >> lg_bits);
            if (lane == l) value = kNone;
        }
        if (!((kept >> group) & 1)) {
#pragma unroll
            for (int i = 0; i < EPL; i++) key[i] = kNone;
        }
    }
    int mine = -1;
    for (int j = 0; j < p.top_k; j++) {
        const float m = max64(key[0]);
        const uint64_t at = __ballot(key[0] == m && m != kNone);
        if (!at) break;
        const int l = __ffsll((unsigned long long)at) - 1;
        const int e = __builtin_amdgcn_readlane(idx[0], l);
        if (lane == j) mine = e;
        if (lane == l) {
#pragma unroll
            for (int i = 0; i + 1 < EPL; i++) {
                key[i] = key[i + 1];
                idx[i] = idx[i + 1];
            }
            key[EPL - 1] = kNone;
        }
    }
    float w = 0.0f;
    if (mine >= 0) w = score_of(logit_at(p, t, mine), p.sigmoid, top, rsum);
    if (p.renormalise) {
        const float s = sum64(w);
        w = s > 0.0f ? w / s : 0.0f;
    }
    if (lane < p.top_k) {
        p.experts_out[t * p.top_k + lane] = mine;
        p.weights_out[t * p.top_k + lane] = w * p.scale;
    }
    return mine;
}

// exclusive sums of n values of LDS, by one wavefront; dst may be src
__device__ __forceinline__ void exclusive(const int* src, int* dst, int n, int lane) {
    int carry = 0;
    for (int e0 = 0; e0 < n; e0 += 64) {
        const int c = e0 + lane < n ? src[e0 + lane] : 0;
        int s = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(s, o, 64);
            if (lane >= o) s += u;
        }
        if (e0 + lane < n) dst[e0 + lane] = carry + s - c;
        carry += __shfl(s, 63, 64);
    }
}

// Places slots [first, last) of the list behind at[e] of each expert's part (at: this
// wavefront's row, of LDS): 64 at a time, a slot's rank among the lanes of its expert.
template <typename Get>
__device__ __forceinline__ void place(const RouteParams& p, int64_t first, int64_t last, int* at, int lane, Get expert) {
    const int bits = 32 - __builtin_clz(p.experts);
    for (int64_t s0 = first; s0 < last; s0 += 64) {
        const int64_t s = s0 + lane;
        const int e = s < last ? expert(s) : -1;
        uint64_t same = __ballot(e >= 0);
        for (int b = 0; b < bits; b++) {
            const uint64_t ones = __ballot((e >> b) & 1);
            same &= ((e >> b) & 1) ? ones : ~ones;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int to = 0;
        if (e >= 0) to = at[e];
        __builtin_amdgcn_wave_barrier();  // every lane has read before one writes
        if (e >= 0) {
            p.slots[to + rank] = (int32_t)s;
            if (rank == 0) at[e] = to + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

}  // namespace

// Choice for the tokens of one range per workgroup (8 wavefronts), and the range's counts.
template <int EPL>
__global__ void __launch_bounds__(512) route_kernel(RouteParams p, int per_range, int lg_bits) {
    __shared__ int hist[kMaxE + 1];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, E = p.experts;
    for (int e = threadIdx.x; e <= E; e += 512) hist[e] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * per_range, last = min(first + per_range, p.tokens);
    for (int64_t t = first + wave; t < last; t += 8) {
        const int e = choose<EPL>(p, t, lane, lg_bits, p.bias);
        if (p.offsets && lane < p.top_k) atomicAdd(&hist[e < 0 ? E : e], 1);  // a count: any order
    }
    if (!p.offsets) return;
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += 512) p.counts[(int64_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// Slots of `ranges` consecutive ranges per workgroup (16 wavefronts).
__global__ void __launch_bounds__(1024) route_place_kernel(RouteParams p, int nranges, int ranges, int64_t range_slots) {
    __shared__ int before[kMaxE + 1], total[kMaxE + 1], part[16][kMaxE + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
    for (int e = tid; e <= E; e += 1024) {
        before[e] = total[e] = 0;
        for (int w = 0; w < 16; w++) part[w][e] = 0;
    }
    __syncthreads();
    const int r0 = blockIdx.x * ranges;
    for (int e0 = 0; e0 <= E; e0 += 64) {
        const int e = e0 + lane;
        int b = 0, all = 0;
        if (e <= E) {
#pragma unroll 8
            for (int r = wave; r < nranges; r += 16) {
                const int c = p.counts[(int64_t)r * (E + 1) + e];
                all += c;
                b += r < r0 ? c : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&before[e], b);
        }
    }
    const int64_t nslots = p.tokens * p.top_k, first = r0 * range_slots, last = min(first + ranges * range_slots, nslots);
    const int64_t quota = (last - first + 1023) / 1024 * 64;  // slots per wavefront
    const int64_t w0 = min(first + wave * quota, last), w1 = min(w0 + quota, last);
    auto expert = [&](int64_t s) {
        const int e = p.experts_out[s];
        return e < 0 ? E : e;
    };
    for (int64_t s = w0 + lane; s < w1; s += 64) atomicAdd(&part[wave][expert(s)], 1);
    __syncthreads();
    if (wave == 0) exclusive(total, total, E + 1, lane);
    __syncthreads();
    for (int e = tid; e <= E; e += 1024) {
        if (blockIdx.x == 0) p.offsets[e] = total[e];
        int at = total[e] + before[e];
        for (int w = 0; w < 16; w++) {
            const int c = part[w][e];
            part[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    place(p, w0, w1, part[wave], lane, expert);
}

// Few tokens: choice and layout in one workgroup (16 wavefronts).
template <int EPL>
__global__ void __launch_bounds__(1024) route_small_kernel(RouteParams p, int lg_bits) {
    __shared__ int part[16][kMaxE + 1], total[kMaxE + 1];
    __shared__ int chosen[kSmallSlots];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
    if (p.offsets) {
        for (int e = tid; e <= E; e += 1024)
            for (int w = 0; w < 16; w++) part[w][e] = 0;
        __syncthreads();
    }
    // a wavefront takes consecutive tokens, so its slots are consecutive too
    const int T = (int)p.tokens, per = (T + 15) / 16, t0 = min(wave * per, T), t1 = min(t0 + per, T);
    for (int t = t0; t < t1; t++) {
        const int e = choose<EPL>(p, t, lane, lg_bits, p.bias);
        if (p.offsets && lane < p.top_k) {
            chosen[t * p.top_k + lane] = e < 0 ? E : e;
            atomicAdd(&part[wave][e < 0 ? E : e], 1);
        }
    }
    if (!p.offsets) return;
    __syncthreads();
    for (int e = tid; e <= E; e += 1024) {
        int n = 0;
        for (int w = 0; w < 16; w++) n += part[w][e];
        total[e] = n;
    }
    __syncthreads();
    if (wave == 0) exclusive(total, total, E + 1, lane);
    __syncthreads();
    for (int e = tid; e <= E; e += 1024) {
        int at = total[e];
        p.offsets[e] = at;
        for (int w = 0; w < 16; w++) {
            const int c = part[w][e];
            part[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    place(p, (int64_t)t0 * p.top_k, (int64_t)t1 * p.top_k, part[wave], lane, [&](int64_t s) { return chosen[s]; });
}

// no tokens: all offsets 0
__global__ void route_empty_kernel(int32_t* offsets, int n) {
    const int i = blockIdx.x * 256 + threadIdx.x;
    if (i < n) offsets[i] = 0;
}

static bool route_small(int64_t tokens, int top_k) { return tokens <= kSmallTokens && tokens * top_k <= kSmallSlots; }

// tokens per range: at most kRanges ranges, of at least 16 tokens
static int64_t route_range(int64_t tokens) {
    const int64_t r = (tokens + kRanges - 1) / kRanges;
    return r < 16 ? 16 : r;
}

size_t route_workspace_bytes(int64_t tokens, int32_t experts, int32_t top_k) {
    if (route_small(tokens, top_k)) return 0;
    const int64_t per = route_range(tokens);
    return (size_t)((tokens + per - 1) / per) * (size_t)(experts + 1) * sizeof(int32_t);
}

template <int EPL>
static hipError_t launch_choice(const RouteParams& p, int lg_bits, hipStream_t s) {
    if (route_small(p.tokens, p.top_k)) {
        const int waves = p.offsets || p.tokens >= 16 ? 16 : (int)p.tokens;
        route_small_kernel<EPL><<<1, 64 * (p.offsets ? 16 : waves), 0, s>>>(p, lg_bits);
        return hipGetLastError();
    }
    const int64_t per = route_range(p.tokens), nranges = (p.tokens + per - 1) / per;
    route_kernel<EPL><<<(unsigned)nranges, 512, 0, s>>>(p, (int)per, lg_bits);
    if (p.offsets) {
        const int64_t nslots = p.tokens * p.top_k;
        int64_t wgs = (nslots + 2047) / 2048;
        if (wgs > 64) wgs = 64;
        const int64_t ranges = (nranges + wgs - 1) / wgs;
        route_place_kernel<<<(unsigned)((nranges + ranges - 1) / ranges), 1024, 0, s>>>(p, (int)nranges, (int)ranges, per * p.top_k);
    }
    return hipGetLastError();
}

hipError_t launch_route(const RouteParams& p, hipStream_t s) {
    if (p.tokens == 0) {
        route_empty_kernel<<<(p.experts + 256) / 256, 256, 0, s>>>(p.offsets, p.experts + 1);
        return hipGetLastError();
    }
    // lanes per group: the largest power of two that gives every group its lanes
    int lg_bits = 6;
    while ((p.groups << lg_bits) > 64) lg_bits--;
    const int lanes = 1 << lg_bits, epl = (p.experts / p.groups + lanes - 1) / lanes;
    if (epl <= 1) return launch_choice<1>(p, lg_bits, s);
    if (epl <= 2) return launch_choice<2>(p, lg_bits, s);
    if (epl <= 4) return launch_choice<4>(p, lg_bits, s);
    if (epl <= 8) return launch_choice<8>(p, lg_bits, s);
    if (epl <= 16) return launch_choice<16>(p, lg_bits, s);
    return launch_choice<32>(p, lg_bits, s);
}

}  // namespace fp4
