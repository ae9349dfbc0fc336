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
// Bound by the vector instructions of the selection: 16384 tokens of 256 experts in 8 groups
// 26.3 us, 19 of them the choice, which issues 476 vector instructions a token, 76 % of the
// cycles of every SIMD (a round of the top_k is about 20: six fused maxima across the lanes,
// the winner's lane by a ballot, the lists' shift by bitwise selects; float maxima, which
// canonicalize, and array selects took 4 us more).  The placement's 8 us are launch, the table
// of counts and the order inside each workgroup.  One token of 64 experts: 4.2 us, 6.5 with the
// call.
#include "fp4_device.h"
#include "layer_internal.h"

namespace fp4 {

namespace {

constexpr int kNone = INT32_MIN;    // key of an expert that cannot be chosen
constexpr int kMaxE = 1024;
constexpr int kRanges = 256;        // ranges of tokens counted apart, at most
// one workgroup routes and places these, two tokens a wavefront (one workgroup / two kernels, us,
// 8 of 64 experts: 16 tokens 6.0 / 8.0, 32 8.0 / 8.3, 48 10.1 / 8.5; 8 of 256: 32 tokens 10.2 / 9.8)
constexpr int kSmallSlots = 1024, kSmallTokens = 32;
constexpr int kKept = 128;           // slots of a wavefront that the placement keeps in LDS
constexpr float kLog2e = 0x1.715476p+0f;

// Keys are compared as integers in the order of their floats (-0 as 0): one instruction per
// step of a maximum.  Its inverse gives the float back.
__device__ __forceinline__ int ordered(float v) {
    const int b = __float_as_int(v + 0.0f);
    return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float unordered(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// v of the lane that a DPP control names
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ int dpp_max(int v) {  // lanes without a source keep v
    return max(v, __builtin_amdgcn_update_dpp(kNone, v, CTRL, 0xF, 0xF, false));
}

// largest v of the wavefront, uniform
__device__ __forceinline__ int max64(int v) {
    v = dpp_max<0xB1>(v);   // neighbours
    v = dpp_max<0x4E>(v);   // pairs
    v = dpp_max<0x141>(v);  // halves of 8
    v = dpp_max<0x140>(v);  // halves of 16
    v = dpp_max<0x142>(v);  // row 0 into 1, 2 into 3
    v = dpp_max<0x143>(v);  // rows 0, 1 into 2, 3
    return __builtin_amdgcn_readlane(v, 63);
}

// sum of v over the wavefront, uniform
__device__ __forceinline__ float sum64(float v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// sum of v over this lane and those below
__device__ __forceinline__ int scan64(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);  // row shifts by 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// the two largest of this lane's (a, b) and those of the lane that a DPP control names
template <int CTRL>
__device__ __forceinline__ void merge2(int& a, int& b) {
    const int c = __builtin_amdgcn_update_dpp(0, a, CTRL, 0xF, 0xF, false);
    const int d = __builtin_amdgcn_update_dpp(0, b, CTRL, 0xF, 0xF, false);
    b = max(min(a, c), max(b, d));
    a = max(a, c);
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

// A lane's part of a wavefront's work: its experts base .. base + count - 1 and their biases.
template <int EPL>
struct Lane {
    int lane, group, place, base, count;
    float bias[EPL];

    __device__ __forceinline__ Lane(const RouteParams& p, int lg_bits) {
        lane = threadIdx.x & 63;
        const int size = p.experts / p.groups;
        group = lane >> lg_bits;
        place = (lane & ((1 << lg_bits) - 1)) * EPL;  // within the group
        base = group * size + place;
        count = group < p.groups ? max(min(size - place, EPL), 0) : 0;
#pragma unroll
        for (int i = 0; i < EPL; i++) bias[i] = p.bias && i < count ? p.bias[base + i] : 0.0f;
    }
};

constexpr int values_per_load(int epl) { return epl % 4 == 0 ? 4 : epl % 2 == 0 ? 2 : 1; }

// this lane's logits of token t (`whole`: its run is one aligned load)
template <int EPL>
__device__ __forceinline__ void load_logits(const RouteParams& p, const Lane<EPL>& me, int64_t t, bool whole, float (&v)[EPL]) {
    if (whole) {
#pragma unroll
        for (int i = 0; i < EPL; i++) v[i] = INFINITY;
        if (me.count == EPL) {
            const int64_t at = t * p.ld + me.base;
            constexpr int W = values_per_load(EPL);
            if (p.logits_bf16) {
                struct alignas(2 * W) Part { uint16_t v[W]; };
                const Part* q = reinterpret_cast<const Part*>(reinterpret_cast<const uint16_t*>(p.logits) + at);
#pragma unroll
                for (int i = 0; i < EPL; i++) v[i] = bf16_bits_to_float(q[i / W].v[i % W]);
            } else {
                struct alignas(4 * W) Part { float v[W]; };
                const Part* q = reinterpret_cast<const Part*>(reinterpret_cast<const float*>(p.logits) + at);
#pragma unroll
                for (int i = 0; i < EPL; i++) v[i] = q[i / W].v[i % W];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < EPL; i++) v[i] = i < me.count ? logit_at(p, t, me.base + i) : INFINITY;
    }
}

// The choice for token t, written out; lane j < top_k returns the j-th expert (or -1).
template <int EPL>
__device__ __forceinline__ int choose(const RouteParams& p, int64_t t, const Lane<EPL>& me, const float (&logit)[EPL], int lg_bits) {
    const int lane = me.lane, group = me.group;
    int key[EPL], idx[EPL];
    int best = kNone;
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        // infinite or NaN: not usable
        key[i] = fabsf(logit[i]) < INFINITY ? ordered(logit[i]) : kNone;
        idx[i] = me.base + i;
        best = max(best, key[i]);
    }
    float top = 0.0f, rsum = 0.0f;
    if (!p.sigmoid) {
        top = unordered(max64(best));
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; i++) s += key[i] == kNone ? 0.0f : __builtin_amdgcn_exp2f(kLog2e * (unordered(key[i]) - top));
        rsum = 1.0f / sum64(s);
    }
    // Keys: score + bias; without a bias the logit, which has the scores' order and neither
    // rounds nor underflows.  A bias of -inf or NaN takes its expert out.
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const float v = score_of(logit[i], p.sigmoid, top, rsum) + me.bias[i];
            key[i] = key[i] != kNone && v > -INFINITY ? ordered(v) : kNone;
        }
    }
#pragma unroll
    for (int a = 0; a + 1 < EPL; a++) {  // largest first; equal keys stay in order
#pragma unroll
        for (int b = EPL - 1; b > a; b--) {
            const bool swap = key[b] > key[b - 1];
            const int k = key[b], x = idx[b];
            key[b] = min(k, key[b - 1]);
            key[b - 1] = max(k, key[b - 1]);
            idx[b] = swap ? idx[b - 1] : x;
            idx[b - 1] = swap ? x : idx[b - 1];
        }
    }
    if (p.groups > 1) {
        // the group's two best values, in all of its lanes
        int a = key[0], b = EPL > 1 ? key[EPL > 1 ? 1 : 0] : kNone;
        if (!p.bias) {
            if (a != kNone) a = ordered(score_of(unordered(a), p.sigmoid, top, rsum));
            if (b != kNone) b = ordered(score_of(unordered(b), p.sigmoid, top, rsum));
        }
        // steps of 1, 2, 4 and 8 lanes (a mirrored half of equal values serves as the step)
        if (lg_bits > 0) merge2<0xB1>(a, b);
        if (lg_bits > 1) merge2<0x4E>(a, b);
        if (lg_bits > 2) merge2<0x141>(a, b);
        if (lg_bits > 3) merge2<0x140>(a, b);
        if (lg_bits > 4) {  // two groups: a 32-lane half each
            const int c = __shfl_xor(a, 16, 64), d = __shfl_xor(b, 16, 64);
            b = max(min(a, c), max(b, d));
            a = max(a, c);
        }
        int value = p.group_top == 2 && b != kNone ? ordered(unordered(a) + unordered(b)) : a;
        if (me.place != 0 || group >= p.groups) value = kNone;
        uint64_t kept = 0;
        for (int j = 0; j < p.top_groups; j++) {
            const int m = max64(value);
            if (m == kNone) break;
            const int l = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(value == m)) - 1;
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
        const int m = max64(key[0]);
        if (m == kNone) break;
        const int l = __ffsll((unsigned long long)__builtin_amdgcn_ballot_w64(key[0] == m)) - 1;
        const int e = __builtin_amdgcn_readlane(idx[0], l);
        mine = lane == j ? e : mine;
        // its lane moves on (bitwise selects: one instruction each)
        const int taken = lane == l ? -1 : 0;
#pragma unroll
        for (int i = 0; i + 1 < EPL; i++) {
            key[i] = (key[i + 1] & taken) | (key[i] & ~taken);
            idx[i] = (idx[i + 1] & taken) | (idx[i] & ~taken);
        }
        key[EPL - 1] = (kNone & taken) | (key[EPL - 1] & ~taken);
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

// total[0 .. n) -> its exclusive sums, by 16 wavefronts (n <= 1025; `chunk`: LDS)
__device__ __forceinline__ void exclusive(int* total, int* chunk, int n) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int c = tid < n ? total[tid] : 0, s = scan64(c);
    if (lane == 63) chunk[wave] = s;
    __syncthreads();
    int carry = 0;
    for (int w = 0; w < wave; w++) carry += chunk[w];
    if (tid < n) total[tid] = carry + s - c;
    if (tid == 1023 && n == 1025) total[1024] = carry + s;
    __syncthreads();
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

// Choice for the tokens of one range per workgroup (16 wavefronts), and the range's counts:
// a row of `stride` values, zeros past the experts.
template <int EPL>
__global__ void __launch_bounds__(1024) route_kernel(RouteParams p, int per_range, int lg_bits, int stride, bool whole) {
    __shared__ int hist[kMaxE];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Lane<EPL> me(p, lg_bits);
    if (threadIdx.x < stride) hist[threadIdx.x] = 0;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * per_range, last = min(first + per_range, p.tokens);
    float next[EPL];
    if (first + wave < last) load_logits<EPL>(p, me, first + wave, whole, next);
    for (int64_t t = first + wave; t < last; t += 16) {
        float logit[EPL];
#pragma unroll
        for (int i = 0; i < EPL; i++) logit[i] = next[i];
        if (t + 16 < last) load_logits<EPL>(p, me, t + 16, whole, next);
        const int e = choose<EPL>(p, t, me, logit, lg_bits);
        if (e >= 0) atomicAdd(&hist[e], 1);  // a count: any order
    }
    if (!p.offsets) return;
    __syncthreads();
    if (threadIdx.x < stride) p.counts[(int64_t)blockIdx.x * stride + threadIdx.x] = hist[threadIdx.x];
}

// Slots of `ranges` consecutive ranges per workgroup (16 wavefronts).
__global__ void __launch_bounds__(1024) route_place_kernel(RouteParams p, int nranges, int ranges, int64_t range_slots, int stride) {
    __shared__ int before[kMaxE + 1], total[kMaxE + 1], chunk[16];
    __shared__ int part[16][kMaxE + 1], list[16][kKept];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
    for (int e = tid; e <= E; e += 1024) before[e] = total[e] = 0;
    for (int e = lane; e <= E; e += 64) part[wave][e] = 0;
    __syncthreads();
    const int r0 = blockIdx.x * ranges;
    const int64_t nslots = p.tokens * p.top_k, first = r0 * range_slots, last = min(first + ranges * range_slots, nslots);
    const int64_t quota = (last - first + 1023) / 1024 * 64;  // slots per wavefront
    const int64_t w0 = min(first + wave * quota, last), w1 = min(w0 + quota, last);
    auto expert = [&](int64_t s) {
        const int e = p.experts_out[s];
        return e < 0 ? E : e;
    };
    // a short list's experts stay in LDS: read once, on their way beside the counts
    const bool kept = quota <= kKept;
    int mine[kKept / 64];
    if (kept) {
#pragma unroll
        for (int i = 0; i < kKept / 64; i++) mine[i] = w0 + 64 * i + lane < w1 ? expert(w0 + 64 * i + lane) : -1;
    }
    int sum = 0;
    for (int e = lane * 4; e < stride; e += 256) {
        int4 all = make_int4(0, 0, 0, 0), b = all;
#pragma unroll 16
        for (int r = wave; r < nranges; r += 16) {
            const int4 c = *reinterpret_cast<const int4*>(p.counts + (int64_t)r * stride + e);
            const int in = r < r0 ? -1 : 0;
            all.x += c.x, all.y += c.y, all.z += c.z, all.w += c.w;
            b.x += c.x & in, b.y += c.y & in, b.z += c.z & in, b.w += c.w & in;
        }
        const int va[4] = {all.x, all.y, all.z, all.w}, vb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (e + i < E) {
                atomicAdd(&total[e + i], va[i]);
                atomicAdd(&before[e + i], vb[i]);
                sum += vb[i];
            }
        }
    }
    sum = scan64(sum);
    if (lane == 63) atomicSub(&before[E], sum);
    if (kept) {
#pragma unroll
        for (int i = 0; i < kKept / 64; i++) {
            list[wave][64 * i + lane] = mine[i];
            if (mine[i] >= 0) atomicAdd(&part[wave][mine[i]], 1);
        }
    } else {
        for (int64_t s = w0 + lane; s < w1; s += 64) atomicAdd(&part[wave][expert(s)], 1);
    }
    __syncthreads();
    exclusive(total, chunk, E + 1);
    for (int e = tid; e <= E; e += 1024) {
        if (blockIdx.x == 0) p.offsets[e] = total[e];
        // slots without an expert: those before the range that no expert has
        int at = total[e] + before[e] + (e == E ? (int)first : 0);
#pragma unroll
        for (int w = 0; w < 16; w++) {
            const int c = part[w][e];
            part[w][e] = at;
            at += c;
        }
    }
    __syncthreads();
    if (kept) place(p, w0, w1, part[wave], lane, [&](int64_t s) { return list[wave][s - w0]; });
    else place(p, w0, w1, part[wave], lane, expert);
}

// Few tokens: choice and layout in one workgroup (16 wavefronts).
template <int EPL>
__global__ void __launch_bounds__(1024) route_small_kernel(RouteParams p, int lg_bits, bool whole) {
    __shared__ int part[16][kMaxE + 1], total[kMaxE + 1], chunk[16];
    __shared__ int chosen[kSmallSlots];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, E = p.experts;
    if (p.offsets)  // a wavefront's own counts
        for (int e = lane; e <= E; e += 64) part[wave][e] = 0;
    // a wavefront takes consecutive tokens, so its slots are consecutive too
    const Lane<EPL> me(p, lg_bits);
    const int T = (int)p.tokens, per = (T + 15) / 16, t0 = min(wave * per, T), t1 = min(t0 + per, T);
    for (int t = t0; t < t1; t++) {
        float logit[EPL];
        load_logits<EPL>(p, me, t, whole, logit);
        const int e = choose<EPL>(p, t, me, logit, lg_bits);
        if (p.offsets && lane < p.top_k) {
            chosen[t * p.top_k + lane] = e < 0 ? E : e;
            atomicAdd(&part[wave][e < 0 ? E : e], 1);
        }
    }
    if (!p.offsets) return;
    __syncthreads();
    for (int e = tid; e <= E; e += 1024) {
        int n = 0;
#pragma unroll
        for (int w = 0; w < 16; w++) n += part[w][e];
        total[e] = n;
    }
    __syncthreads();
    exclusive(total, chunk, E + 1);
    for (int e = tid; e <= E; e += 1024) {
        int at = total[e];
        p.offsets[e] = at;
#pragma unroll
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

static int route_stride(int experts) { return (experts + 3) & ~3; }

size_t route_workspace_bytes(int64_t tokens, int32_t experts, int32_t top_k) {
    if (route_small(tokens, top_k)) return 0;
    const int64_t per = route_range(tokens);
    return (size_t)((tokens + per - 1) / per) * (size_t)route_stride(experts) * sizeof(int32_t);
}

template <int EPL>
static hipError_t launch_choice(const RouteParams& p, int lg_bits, hipStream_t s) {
    // whether every lane's run of experts is whole and aligned for one load (of 16 bytes at most)
    constexpr int W = values_per_load(EPL);
    const int size = p.experts / p.groups, bytes = (p.logits_bf16 ? 2 : 4) * W;
    const bool whole = W > 1 && size % EPL == 0 && p.ld % W == 0 && reinterpret_cast<uintptr_t>(p.logits) % bytes == 0;

    if (route_small(p.tokens, p.top_k)) {
        const int waves = p.offsets || p.tokens >= 16 ? 16 : (int)p.tokens;
        route_small_kernel<EPL><<<1, 64 * waves, 0, s>>>(p, lg_bits, whole);
        return hipGetLastError();
    }
    const int64_t per = route_range(p.tokens), nranges = (p.tokens + per - 1) / per;
    route_kernel<EPL><<<(unsigned)nranges, 1024, 0, s>>>(p, (int)per, lg_bits, route_stride(p.experts), whole);
    if (p.offsets) {
        const int64_t nslots = p.tokens * p.top_k;
        // A workgroup per 512 slots, of whole ranges (512 / 1024 / 2048 slots with at most 256
        // workgroups, and 2048 with 64, us for choice and placement: 256 tokens of 64 experts, 8
        // each, 9.4 / 9.5 / 10.3 / 10.3; 4096 of 256 13.3 / 13.6 / 14.5 / 14.5; 65536 of 64
        // 44.1 / 44.3 / 44.2 / 50.4).
        const int64_t wgs = min((nslots + 511) / 512, nranges);
        const int64_t ranges = (nranges + wgs - 1) / wgs;
        route_place_kernel<<<(unsigned)((nranges + ranges - 1) / ranges), 1024, 0, s>>>(p, (int)nranges, (int)ranges, per * p.top_k,
                                                                                           route_stride(p.experts));
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
    if (epl <= 3) return launch_choice<3>(p, lg_bits, s);
    if (epl <= 4) return launch_choice<4>(p, lg_bits, s);
    if (epl <= 6) return launch_choice<6>(p, lg_bits, s);
    if (epl <= 8) return launch_choice<8>(p, lg_bits, s);
    if (epl <= 12) return launch_choice<12>(p, lg_bits, s);
    if (epl <= 16) return launch_choice<16>(p, lg_bits, s);
    return launch_choice<32>(p, lg_bits, s);
}

}  // namespace fp4
