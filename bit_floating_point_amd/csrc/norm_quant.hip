// Rows of activations to 8-bit codes: the residual addition with the root-mean-square
// norm, SwiGLU, and the 128 x 128 blocks of weights.
//
// All three are one pass over HBM, which bounds them.  A lane owns 8 consecutive columns (one
// 16-byte load of bf16, two of binary32, one 8-byte store of codes); a row stays in registers
// between its reduction and its output, so every value is read once.  Inputs are read
// nontemporally (nothing reads them again).  Sums, statistics and scales are binary32; codes
// round once, from binary32.
//
// Measured (us, bytes of inputs and outputs over time): norm of 4096 x 5120 with eight
// weighted bf16 terms, residual, codes per 128 and bf16 rows 87 (5.5 TB/s); with one term and no
// rows 34 (4.3); 777 x 11016 f32 with a static scale 30.5 (3.6); one row of 5120 3.7 in the kernel, 8
// with the call; 2^18 rows of 512, one wavefront each, 153 (6.2), but 2^20 rows of 128, which fill
// 16 of its lanes, 386 (1.0).  SwiGLU 4096 x 13824 47 (6.1 TB/s), with row scales 54 (5.3).  Block
// weights 15360 x 5120 bf16 50 (4.8), f32 74 (5.3); 32 of 4096 x 5120 bf16 377 (5.3).  A copy on
// this card reaches 4.8 TB/s, reads 6.
#include <type_traits>

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

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false));
}
// sum over the wavefront, in lane 63
__device__ __forceinline__ float wave_sum(float v) {
    v = dpp_add<0xB1>(v);        // neighbours
    v = dpp_add<0x4E>(v);        // pairs
    v = dpp_add<0x141>(v);       // halves of 8
    v = dpp_add<0x140>(v);       // halves of 16
    v = dpp_add<0x142, 0xA>(v);  // row 0 into 1, 2 into 3
    v = dpp_add<0x143, 0xC>(v);  // rows 0, 1 into 2, 3
    return v;
}

// Sum over a row: v[c] is this lane's part of chunk segment c waves + w (64 chunks of 8
// columns each).  Segments are summed apart and then added in order (by sixteens), so the result does not
// depend on how many of them a wavefront holds, that is on the number of rows.
template <int NC>
__device__ __forceinline__ float row_sum(const float (&v)[NC], float* part, int waves, int segments) {
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const float s = wave_sum(v[c]);
        if ((threadIdx.x & 63) == 63) part[c * waves + wave] = s;
    }
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < segments; i += 16) {
        float u = part[i];
        for (int k = i + 1; k < min(i + 16, segments); k++) u += part[k];
        t += u;
    }
    return t;
}
// Maximum over the wavefronts of a workgroup; `part` holds one value per wavefront.  Every
// lane returns the result.
__device__ __forceinline__ float block_max(float v, float* part, int waves) {
    v = wave_max(v);
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    float t = 0.0f;
    for (int i = 0; i < waves; i++) t = fmaxf(t, part[i]);
    return t;
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

// A unit's scale s = fl32(amax / Qmax), rounded to binary16 where scales are stored so: a
// product and a correction, correctly rounded unless subnormal (checked likewise).
__device__ __forceinline__ float unit_scale(float amax, const CodeOut& o) {
    float s;
    if (amax >= 0x1p-100f && amax <= 0x1p120f) {
        const float q = amax * o.rqmax;
        s = __builtin_fmaf(__builtin_fmaf(-q, o.qmax, amax), o.rqmax, q);
    } else {
        s = amax > 0.0f ? fmaxf(amax / o.qmax, kLeastScale) : 0.0f;
    }
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
            y[i] = v[i] * fminf(ldexpf(r, -sh), kLargest);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = v[i] * r;
    }
    // a unit's own binary32 scale (never below kLeastScale) keeps its values within half a step
    // of Qmax; a given scale does not, nor one that binary16 rounded
    if (o.mode == 0 || o.scale_f16) {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __builtin_amdgcn_fmed3f(y[i], -o.qmax, o.qmax);
    }
    *reinterpret_cast<uint2*>(o.packed + row * o.ldp + col) = codes8(y, o.e4m3);
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
        r = reciprocal(s);
    } else if (o.mode == 0) {
        r = reciprocal(*o.tensor_scale);
    }
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (o.mode == 2) {
            const float s = unit_scale(lanes_max(amax8(v[c]), o.group / 8), o);
            if (col < cols && col % o.group == 0) store_unit_scale(o, row * ((cols + o.group - 1) / o.group) + col / o.group, s);
            r = reciprocal(s);
        }
        if (col < cols) store_codes8(o, row, col, v[c], r);
    }
}

}  // namespace

// One workgroup per row; NC chunks of 8 columns per thread.
template <int NC, bool XBF>
__global__ void __launch_bounds__(1024) rmsnorm_quant_kernel(NormParams p) {
    __shared__ float sums[128], part[16];
    const int waves = (int)(blockDim.x >> 6);
    const int64_t row = blockIdx.x;
    float h[NC][8];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
#pragma unroll
        for (int i = 0; i < 8; i++) h[c][i] = 0.0f;
        if (p.residual && col < p.cols) get8<true>(p.residual, p.residual_bf16, row * p.ldr + col, h[c]);
    }
    // U terms at a time, their loads together; an absent term's row may hold anything: its
    // values are dropped
    constexpr int U = NC <= 2 ? 4 : 1;
    auto add = [&](int j, auto count) {
        constexpr int C = decltype(count)::value;
        float w[C];
#pragma unroll
        for (int q = 0; q < C; q++) w[q] = p.term_weights ? p.term_weights[row * p.terms + j + q] : 1.0f;
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
            float x[C][8];
            if (col < p.cols) {
#pragma unroll
                for (int q = 0; q < C; q++) get8<true>(p.x, XBF, (row * p.terms + j + q) * p.ldx + col, x[q]);
#pragma unroll
                for (int q = 0; q < C; q++)
#pragma unroll
                    for (int i = 0; i < 8; i++) h[c][i] = w[q] != 0.0f ? __builtin_fmaf(w[q], x[q][i], h[c][i]) : h[c][i];
            }
        }
    };
    int j = 0;
    for (; j + U <= p.terms; j += U) add(j, std::integral_constant<int, U>{});
    for (; j < p.terms; j++) add(j, std::integral_constant<int, 1>{});
    float ss[NC];
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (p.residual_out && col < p.cols) put8(p.residual_out, p.residual_bf16, row * p.ldro + col, h[c]);
        ss[c] = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; i++) ss[c] = __builtin_fmaf(h[c][i], h[c][i], ss[c]);
    }
    if (!p.out.packed && !p.y) return;
    float g[NC][8];  // on its way while the sum is reduced
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (NC <= 2 && col < p.cols) get8(p.gamma, p.gamma_bf16, col, g[c]);
    }
    const float rstd = 1.0f / sqrtf(row_sum<NC>(ss, sums, waves, (int)((p.cols + 511) / 512)) / (float)p.cols + p.eps);
#pragma unroll
    for (int c = 0; c < NC; c++) {
        const int64_t col = ((int64_t)c * blockDim.x + threadIdx.x) * 8;
        if (col < p.cols) {
            if (NC > 2) get8(p.gamma, p.gamma_bf16, col, g[c]);
#pragma unroll
            for (int i = 0; i < 8; i++) h[c][i] = (h[c][i] * rstd) * g[c][i];
            if (p.y) put8(p.y, p.y_bf16, row * p.ldy + col, h[c]);
        }
    }
    if (p.out.packed) emit_row<NC>(p.out, row, p.cols, h, part, waves);
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
            get8<true>(p.x, p.x_bf16, row * p.ldx + col, g);
            get8<true>(p.x, p.x_bf16, row * p.ldx + p.cols + col, u);
#pragma unroll
            for (int i = 0; i < 8; i++) h[c][i] = swiglu(g[i], u[i]);
        }
    }
    emit_row<NC>(p.out, row, p.cols, h, part, (int)(blockDim.x >> 6));
}

// The same without per-row scales, where no reduction crosses a wavefront: a workgroup of
// 256 threads takes 2^cbits chunks (of 8 columns) of 256 / 2^cbits rows.
template <bool XBF>
__global__ void __launch_bounds__(256) swiglu_quant_flat_kernel(SwigluParams p, int cbits, uint32_t parts) {
    const uint32_t part = blockIdx.x % parts, rows = blockIdx.x / parts;
    const int64_t row = (int64_t)rows * (256 >> cbits) + (threadIdx.x >> cbits);
    const int64_t col = ((int64_t)part * (1 << cbits) + (threadIdx.x & ((1 << cbits) - 1))) * 8;
    const bool in = row < p.rows && col < p.cols;
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; i++) h[i] = 0.0f;
    if (in) {
        float g[8], u[8];
        get8<true>(p.x, XBF, row * p.ldx + col, g);
        get8<true>(p.x, XBF, row * p.ldx + p.cols + col, u);
#pragma unroll
        for (int i = 0; i < 8; i++) h[i] = swiglu(g[i], u[i]);
    }
    float r;
    if (p.out.mode == 2) {
        const float s = unit_scale(lanes_max(amax8(h), p.out.group / 8), p.out);
        if (in && col % p.out.group == 0)
            store_unit_scale(p.out, row * ((p.cols + p.out.group - 1) / p.out.group) + col / p.out.group, s);
        r = reciprocal(s);
    } else {
        r = reciprocal(*p.out.tensor_scale);
    }
    if (in) store_codes8(p.out, row, col, h, r);
}

// One workgroup per block of 128 x 128: thread t holds 8 columns of rows t / 16 + 16 i.
template <bool BF16>
__global__ void __launch_bounds__(256) quantize_block_kernel(BlockQuantParams p, int64_t first, int nb, int kb) {
    __shared__ float part[4];
    const int64_t b = first + blockIdx.x;
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
    const float top = block_max(amax, part, 4);
    const float s = top > 0.0f ? fmaxf(top / p.qmax, kLeastScale) : 0.0f;
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

// p advanced by `bytes` (null stays null)
template <typename T>
static T* ahead(T* p, int64_t bytes) {
    return p ? reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes) : p;
}

// the outputs, and the operands, of rows first .. first + rows - 1
static CodeOut rows_of(const CodeOut& o, int64_t cols, int64_t first) {
    CodeOut q = o;
    const int64_t units = o.mode == 1 ? 1 : o.mode == 2 ? (cols + o.group - 1) / o.group : 0;
    q.packed = ahead(o.packed, first * o.ldp);
    q.scales = ahead(o.scales, first * units * (o.scale_f16 ? 2 : 4));
    return q;
}
static NormParams rows_of(const NormParams& p, int64_t first, int64_t rows) {
    NormParams q = p;
    const int64_t stream = p.residual_bf16 ? 2 : 4;
    q.rows = rows;
    q.x = ahead(p.x, first * p.terms * p.ldx * (p.x_bf16 ? 2 : 4));
    q.term_weights = ahead(p.term_weights, first * p.terms * 4);
    q.residual = ahead(p.residual, first * p.ldr * stream);
    q.residual_out = ahead(p.residual_out, first * p.ldro * stream);
    q.y = ahead(p.y, first * p.ldy * (p.y_bf16 ? 2 : 4));
    q.out = rows_of(p.out, p.cols, first);
    return q;
}
static SwigluParams rows_of(const SwigluParams& p, int64_t first, int64_t rows) {
    SwigluParams q = p;
    q.rows = rows;
    q.x = ahead(p.x, first * p.ldx * (p.x_bf16 ? 2 : 4));
    q.out = rows_of(p.out, p.cols, first);
    return q;
}

// `launch` on parts of at most `most` rows
template <typename Params, typename Launch>
static hipError_t by_rows(const Params& p, int64_t most, Launch launch) {
    for (int64_t first = 0; first < p.rows; first += most) {
        launch(p.rows <= most ? p : rows_of(p, first, p.rows - first < most ? p.rows - first : most));
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Chunks per thread.  Few rows, whose latency counts: one (64 x 8192 of 8 terms: 9.4 us against
// 14.9 with two).  Many: with several terms in flight two (4096 x 5120 of 8 terms, one / two /
// four chunks: 91 / 90 / 98 us), with one term four, so that enough bytes are on their way
// (8192 x 5120 without a residual: 58 / 49 / 41 us; 4096 x 5120: 44 / 39 / 36).
template <bool XBF>
static hipError_t launch_norm(const NormParams& p, hipStream_t s) {
    const int64_t chunks = (p.cols + 7) / 8;
    // (777 x 11016 f32 of one term: two chunks 28 us, four 32)
    const int few = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : chunks <= 4096 ? 4 : 8;
    const int many = chunks <= 256 ? 1 : p.terms > 1 && chunks <= 2048 ? 2 : chunks <= 4096 ? 4 : 8;
    const int nc = p.rows < 1024 ? few : many;
    const int threads = 64 * waves_for(chunks, nc);
    return by_rows(p, max_workgroups(threads), [&](const NormParams& q) {
        const dim3 grid((unsigned)q.rows);
        if (nc == 1) rmsnorm_quant_kernel<1, XBF><<<grid, threads, 0, s>>>(q);
        else if (nc == 2) rmsnorm_quant_kernel<2, XBF><<<grid, threads, 0, s>>>(q);
        else if (nc == 4) rmsnorm_quant_kernel<4, XBF><<<grid, threads, 0, s>>>(q);
        else rmsnorm_quant_kernel<8, XBF><<<grid, threads, 0, s>>>(q);
    });
}

hipError_t launch_rmsnorm_quant(const NormParams& p, hipStream_t s) {
    return p.x_bf16 ? launch_norm<true>(p, s) : launch_norm<false>(p, s);
}

hipError_t launch_swiglu_quant(const SwigluParams& p, hipStream_t s) {
    const int64_t chunks = (p.cols + 7) / 8;
    if (p.out.mode != 1) {
        // whole groups per row: at least the lanes of a group
        int cbits = p.out.mode == 2 && p.out.group > 8 ? __builtin_ctz(p.out.group / 8) : 0;
        while (cbits < 8 && (1 << cbits) < chunks) cbits++;
        const int64_t parts = (chunks + (1 << cbits) - 1) >> cbits, height = 256 >> cbits;  // of a workgroup, in rows
        return by_rows(p, max_workgroups(256) / parts * height, [&](const SwigluParams& q) {
            const unsigned grid = (unsigned)(parts * ((q.rows + height - 1) / height));
            if (q.x_bf16) swiglu_quant_flat_kernel<true><<<grid, 256, 0, s>>>(q, cbits, (uint32_t)parts);
            else swiglu_quant_flat_kernel<false><<<grid, 256, 0, s>>>(q, cbits, (uint32_t)parts);
        });
    }
    // Row scales.  Below 1024 rows a row's latency counts: as few chunks per thread as a workgroup
    // of 1024 covers (one / two / four / eight chunks, us: 512 x 4096 4.8 / 5.6 / 7.6 / 10.8; 512 x
    // 11008 two 8.2, four 9.8; 64 x 32768 four 8.8, eight 12.3).  With more rows their bytes do: two
    // up to 8192 columns (4096 x 8192: 34.8 / 31.6 / 32.9 / 36.4; but one for 2048 and less, 1024 x
    // 2048: 5.1 / 5.8), then four (4096 x 13824 two 60.3, four 54.0, eight 59.6).
    const int few = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : chunks <= 4096 ? 4 : 8;
    const int nc = p.rows < 1024 || chunks <= 256 || chunks > 4096 ? few : chunks <= 1024 ? 2 : 4;
    const int threads = 64 * waves_for(chunks, nc);
    return by_rows(p, max_workgroups(threads), [&](const SwigluParams& q) {
        const dim3 grid((unsigned)q.rows);
        if (nc == 1) swiglu_quant_kernel<1><<<grid, threads, 0, s>>>(q);
        else if (nc == 2) swiglu_quant_kernel<2><<<grid, threads, 0, s>>>(q);
        else if (nc == 4) swiglu_quant_kernel<4><<<grid, threads, 0, s>>>(q);
        else swiglu_quant_kernel<8><<<grid, threads, 0, s>>>(q);
    });
}

hipError_t launch_quantize_block(const BlockQuantParams& p, hipStream_t s) {
    const int64_t nb = (p.n + kBlock - 1) / kBlock, kb = (p.k + kBlock - 1) / kBlock;
    const int64_t blocks = p.batch * nb * kb, most = max_workgroups(256);
    for (int64_t first = 0; first < blocks; first += most) {
        const unsigned grid = (unsigned)(blocks - first < most ? blocks - first : most);
        if (p.bf16) quantize_block_kernel<true><<<grid, 256, 0, s>>>(p, first, (int)nb, (int)kb);
        else quantize_block_kernel<false><<<grid, 256, 0, s>>>(p, first, (int)nb, (int)kb);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace fp4
