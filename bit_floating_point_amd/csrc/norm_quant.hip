// Rows of activations to 8-bit codes: the residual addition with the root-mean-square
// norm, SwiGLU, and the 128 x 128 blocks of weights.
//
// All three are one pass over HBM.  A lane owns 8 consecutive columns (one 16-byte load
// of bf16, two of binary32, one 8-byte store of codes); a row stays in registers between
// its reduction and its output, so every value is read once.  Sums, statistics and
// scales are binary32; codes round once, from binary32.
#include "fp4_device.h"
#include "layer_internal.h"

namespace fp4 {

namespace {

// largest magnitude of eight values
__device__ __forceinline__ float amax8(const float v[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) m = fmaxf(m, fabsf(v[i]));
    return m;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// Reductions over the wavefronts of a workgroup; `part` holds one value per wavefront.
// Every lane returns the result; the caller keeps two reductions of one kernel in
// different arrays, so one barrier each suffices.
__device__ __forceinline__ float block_sum(float v, float* part, int waves) {
    v = wave_sum(v);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < waves; i++) t += part[i];
    return t;
}
__device__ __forceinline__ float block_max(float v, float* part, int waves) {
    v = wave_max(v);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < waves; i++) t = fmaxf(t, part[i]);
    return t;
}

// Eight 8-bit codes of y: clipped to the grid's range, then the hardware's conversion
// (nearest, ties to the even code, sign kept; checked against the oracle's nearest-point
// search).
template <bool E4M3>
__device__ __forceinline__ uint2 codes8(const float y[8]) {
    constexpr float top = E4M3 ? 448.0f : 57344.0f;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; i++) v[i] = __builtin_amdgcn_fmed3f(y[i], -top, top);
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

// s = amax / Qmax, rounded to binary16 where scales are stored so
__device__ __forceinline__ float unit_scale(float amax, const CodeOut& o) {
    const float s = amax / o.qmax;
    return o.scale_f16 ? round_f16(s) : s;
}
__device__ __forceinline__ void store_unit_scale(const CodeOut& o, int64_t unit, float s) {
    if (o.scale_f16) reinterpret_cast<__half*>(o.scales)[unit] = __float2half_rn(s);
    else reinterpret_cast<float*>(o.scales)[unit] = s;
}

// codes of v at columns col .. col + 7 of a row with reciprocal scale r (and 2^-k)
__device__ __forceinline__ void store_codes8(const CodeOut& o, int64_t row, int64_t col, const float v[8], float r) {
    float y[8];
    if (o.col_shift) {
        const uint2 k = *reinterpret_cast<const uint2*>(o.col_shift + col);
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int sh = (int)(int8_t)((i < 4 ? k.x : k.y) >> (8 * (i & 3)));
            y[i] = v[i] * ldexpf(r, -sh);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i] * r;
    }
    *reinterpret_cast<uint2*>(o.packed + row * o.ldp + col) = codes8(y, o.e4m3);
}

// eight values at columns col .. col + 7 of a row of f32 or bf16
__device__ __forceinline__ void get8(const void* base, bool bf16, int64_t at, float v[8]) {
    if (bf16) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + at);
        raw8_to_float<true>(Raw8{u, u}, v);
    } else {
        const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(base) + at);
        raw8_to_float<false>(Raw8{q[0], q[1]}, v);
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

// Codes and scales of the row held as v[NC][8]: chunk c of thread t covers columns
// 8 (c blockDim + t) .. + 7 (values past the row are zeros).  `part`: LDS for one
// reduction over the workgroup.
template <int NC>
__device__ __forceinline__ void emit_row(const CodeOut& o, int64_t row, int64_t cols, const float (&v)[NC][8], float* part,
                                         int waves) {
    float r = 0.0f;
    if (o.mode == 1) {
        float m = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; c++) m = fmaxf(m, amax8(v[c]));
        const float s = unit_scale(block_max(m, part, waves), o);
        if (threadIdx.x == 0) store_unit_scale(o, row, s);
        r = recip_or_zero(s);
    } else if (o.mode == 0) {
        r = recip_or_zero(*o.tensor_scale);
    }
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (o.mode == 2) {
            const float s = unit_scale(group_max(amax8(v[c]), o.group / 8), o);
            if (col < cols && col % o.group == 0) store_unit_scale(o, row * ((cols + o.group - 1) / o.group) + col / o.group, s);
            r = recip_or_zero(s);
        }
        if (col < cols) store_codes8(o, row, col, v[c], r);
    }
}

}  // namespace

// One workgroup per row; NC chunks of 8 columns per thread.
template <int NC>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(NormParams p) {
    __shared__ float part[2][16];
    const int waves = (int)(blockDim.x >> 6);
    const int64_t row = blockIdx.x;
    float h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int i = 0; i < 8; i++) h[c][i] = 0.0f;
        if (p.residual && col < p.cols) get8(p.residual, p.residual_bf16, row * p.ldr + col, h[c]);
    }
    for (int j = 0; j < p.terms; j++) {
        const float w = p.term_weights ? p.term_weights[row * p.terms + j] : 1.0f;
        if (w == 0.0f) continue;  // an absent term: its row may hold anything
        const int64_t at = (row * p.terms + j) * p.ldx;
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
            float x[8];
            if (col < p.cols) {
                get8(p.x, p.x_bf16, at + col, x);
#pragma unroll
                for (int i = 0; i < 8; i++) h[c][i] = __builtin_fmaf(w, x[i], h[c][i]);
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (p.residual_out && col < p.cols) put8(p.residual_out, p.residual_bf16, row * p.ldro + col, h[c]);
#pragma unroll
        for (int i = 0; i < 8; i++) ss = __builtin_fmaf(h[c][i], h[c][i], ss);
    }
    if (!p.out.packed && !p.y) return;
    const float rstd = 1.0f / sqrtf(block_sum(ss, part[0], waves) / (float)p.cols + p.eps);
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (col < p.cols) {
            float g[8];
            get8(p.gamma, p.gamma_bf16, col, g);
#pragma unroll
            for (int i = 0; i < 8; i++) h[c][i] = (h[c][i] * rstd) * g[i];
            if (p.y) put8(p.y, p.y_bf16, row * p.ldy + col, h[c]);
        }
    }
    if (p.out.packed) emit_row<NC>(p.out, row, p.cols, h, part[1], waves);
}

// g / (1 + e^-g) * u: e^x as 2^(x log2 e) and a reciprocal, both the hardware's
__device__ __forceinline__ float swiglu(float g, float u) {
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -0x1.715476p+0f)) * u;
}

template <int NC>
__global__ void __launch_bounds__(1024) swiglu_quant_kernel(SwigluParams p) {
    __shared__ float part[16];
    const int64_t row = blockIdx.x;
    float h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int i = 0; i < 8; i++) h[c][i] = 0.0f;
        if (col < p.cols) {
            float g[8], u[8];
            get8(p.x, p.x_bf16, row * p.ldx + col, g);
            get8(p.x, p.x_bf16, row * p.ldx + p.cols + col, u);
#pragma unroll
            for (int i = 0; i < 8; i++) h[c][i] = swiglu(g[i], u[i]);
        }
    }
    emit_row<NC>(p.out, row, p.cols, h, part, (int)(blockDim.x >> 6));
}

// One workgroup per block of 128 x 128: thread t holds 8 columns of rows t / 16 + 16 i.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_block_kernel(BlockQuantParams p, int nb, int kb) {
    __shared__ float part[4];
    const int64_t b = blockIdx.x;
    const int64_t kblk = b % kb, nblk = (b / kb) % nb, m = b / ((int64_t)kb * nb);
    const int64_t col = kblk * kBlock + (threadIdx.x & 15) * 8;
    float v[8][8], amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t row = nblk * kBlock + (threadIdx.x >> 4) + 16 * i;
#pragma unroll
        for (int j = 0; j < 8; j++) v[i][j] = 0.0f;
        if (row < p.n && col < p.k) get8(p.w, BF16, m * p.stride_w + row * p.ldw + col, v[i]);
        amax = fmaxf(amax, amax8(v[i]));
    }
    const float s = block_max(amax, part, 4) / p.qmax;
    if (threadIdx.x == 0) p.scales[b] = s;
    const float r = recip_or_zero(s);
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t row = nblk * kBlock + (threadIdx.x >> 4) + 16 * i;
        if (row < p.n && col < p.k) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; j++) y[j] = v[i][j] * r;
            *reinterpret_cast<uint2*>(p.packed + m * p.stride_p + row * p.ldp + col) = codes8(y, p.e4m3);
        }
    }
}

// wavefronts of a workgroup that covers `chunks` chunks of 8 columns, nc per thread
static int waves_for(int64_t chunks, int nc) { return (int)((chunks + 64 * nc - 1) / (64 * nc)); }

hipError_t launch_rmsnorm_quant(const NormParams& p, hipStream_t s) {
    const int64_t chunks = (p.cols + 7) / 8;
    const dim3 grid((unsigned)p.rows);
    if (chunks <= 1024) rmsnorm_quant_kernel<1><<<grid, 64 * waves_for(chunks, 1), 0, s>>>(p);
    else if (chunks <= 2048) rmsnorm_quant_kernel<2><<<grid, 64 * waves_for(chunks, 2), 0, s>>>(p);
    else rmsnorm_quant_kernel<8><<<grid, 64 * waves_for(chunks, 8), 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_swiglu_quant(const SwigluParams& p, hipStream_t s) {
    const int64_t chunks = (p.cols + 7) / 8;
    const dim3 grid((unsigned)p.rows);
    if (chunks <= 1024) swiglu_quant_kernel<1><<<grid, 64 * waves_for(chunks, 1), 0, s>>>(p);
    else if (chunks <= 2048) swiglu_quant_kernel<2><<<grid, 64 * waves_for(chunks, 2), 0, s>>>(p);
    else swiglu_quant_kernel<8><<<grid, 64 * waves_for(chunks, 8), 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_quantize_block(const BlockQuantParams& p, hipStream_t s) {
    const int64_t nb = (p.n + kBlock - 1) / kBlock, kb = (p.k + kBlock - 1) / kBlock;
    const dim3 grid((unsigned)(p.batch * nb * kb));
    if (p.bf16) quantize_block_kernel<true><<<grid, 256, 0, s>>>(p, (int)nb, (int)kb);
    else quantize_block_kernel<false><<<grid, 256, 0, s>>>(p, (int)nb, (int)kb);
    return hipGetLastError();
}

}  // namespace fp4
