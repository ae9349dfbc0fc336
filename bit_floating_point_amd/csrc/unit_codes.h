// Eight values at a time between memory, binary32 and 8-bit codes, and the scale of a unit of
// values: what the kernels that quantize rows share.
#pragma once
#include "fp4_device.h"

namespace fp4 {

// largest magnitude of eight values
__device__ __forceinline__ float amax8(const float v[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));
    return m;
}

// largest of v >= 0 over aligned groups of `lanes` lanes (a power of two); numbers that are
// not negative are in the order of their bits
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float lanes_max(float amax, int lanes) {
    uint32_t v = __float_as_uint(amax);
    if (lanes >= 2) v = dpp_max<0xB1>(v);    // neighbours
    if (lanes >= 4) v = dpp_max<0x4E>(v);    // pairs
    if (lanes >= 8) v = dpp_max<0x141>(v);   // halves of 8
    if (lanes >= 16) v = dpp_max<0x140>(v);  // halves of 16
    for (int o = 16; o < lanes; o <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, o, 64));
    return __uint_as_float(v);
}

// Eight 8-bit codes of y by the hardware's conversion (nearest, ties to the even code, sign
// kept; checked against the oracle's nearest-point search).  It saturates nowhere, so values
// that may pass the grid's end are clipped first.
template <bool E4M3>
__device__ __forceinline__ uint2 codes8(const float v[8]) {
    int lo = 0, hi = 0;
    if constexpr (E4M3) {
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
    } else {
        lo = __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], lo, false);
        lo = __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], lo, true);
        hi = __builtin_amdgcn_cvt_pk_bf8_f32(v[4], v[5], hi, false);
        hi = __builtin_amdgcn_cvt_pk_bf8_f32(v[6], v[7], hi, true);
    }
    return make_uint2((uint32_t)lo, (uint32_t)hi);
}
__device__ __forceinline__ uint2 codes8(const float y[8], bool e4m3) { return e4m3 ? codes8<true>(y) : codes8<false>(y); }

constexpr float kLargest = 0x1.fffffep+127f;  // a factor past it would turn zeros into NaN

// fl32(1 / s), 0 for s = 0: the hardware's reciprocal and one Newton step, which is the
// correctly rounded value wherever neither is subnormal (checked for every significand)
__device__ __forceinline__ float reciprocal(float s) {
    if (s >= 0x1p-120f && s <= 0x1p120f) {
        const float r = __builtin_amdgcn_rcpf(s);
        return __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
    }
    return fminf(recip_or_zero(s), kLargest);
}

// The least scale of a unit with a value that is not 0: the smallest normal number.  Below
// 2^-128 a scale has no binary32 reciprocal; with this one such values keep their codes'
// absolute precision, half the smallest code's value times 2^-126.
constexpr float kLeastScale = 0x1p-126f;

// A unit's scale s = fl32(amax / Qmax): a product with rqmax = fl32(1 / Qmax) and a correction,
// correctly rounded unless subnormal (checked likewise).
__device__ __forceinline__ float scale_of(float amax, float qmax, float rqmax) {
    if (amax >= 0x1p-100f && amax <= 0x1p120f) {
        const float q = amax * rqmax;
        return __builtin_fmaf(__builtin_fmaf(-q, qmax, amax), rqmax, q);
    }
    return amax > 0.0f ? fmaxf(amax / qmax, kLeastScale) : 0.0f;
}

// eight values at columns col .. col + 7 of a row of f32 or bf16; ONCE: nothing reads them
// again soon
template <bool ONCE>
__device__ __forceinline__ uint4 get16(const void* p) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4* q = reinterpret_cast<const u32x4*>(p);
    const u32x4 v = ONCE ? __builtin_nontemporal_load(q) : *q;
    return make_uint4(v[0], v[1], v[2], v[3]);
}
template <bool ONCE = false>
__device__ __forceinline__ void get8(const void* base, bool bf16, int64_t at, float v[8]) {
    if (bf16) {
        const uint4 u = get16<ONCE>(reinterpret_cast<const uint16_t*>(base) + at);
        raw8_to_float<true>(Raw8{u, u}, v);
    } else {
        const float* q = reinterpret_cast<const float*>(base) + at;
        raw8_to_float<false>(Raw8{get16<ONCE>(q), get16<ONCE>(q + 4)}, v);
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void put8(void* base, bool bf16, int64_t at, const float v[8]) {
    if (bf16) {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + at) =
            make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    } else {
        float4* q = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + at);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

}  // namespace fp4
