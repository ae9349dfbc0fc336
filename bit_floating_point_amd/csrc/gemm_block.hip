// Products of 8-bit operands whose scales change along K:
//   Y[m, n] = T,  T = fma(P_b[m, n], fl32(sa[m, b] * sw[n / 128, b]), T) over the blocks b
// of 128 columns of K, P_b = sum over the block of the code products on the f8f6f4 matrix
// cores.  The scales differ from block to block, so a block's sum cannot stay in the
// accumulator of the next: every block ends in one fused multiply-add per output value.
//
// The weight tile is the instruction's first operand, so a lane of a 32 x 32 result holds
// 16 columns n of one row m: both scales are one value per lane and block, and four
// consecutive columns leave in one store.
#include "fp4_device.h"
#include "layer_internal.h"

namespace fp4 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int FW, int FA>
__device__ __forceinline__ f32x16 mfma64(i32x8 w, i32x8 a, f32x16 c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, FW, FA, 0, 127, 0, 127);
}

// 32 codes of a row at k .. k + 31, zeros past K (a multiple of 16); `row` null: zeros
__device__ __forceinline__ i32x8 load32(const uint8_t* row, int64_t k, int64_t K) {
    uint4 u = make_uint4(0, 0, 0, 0), v = u;
    if (row && k < K) u = *reinterpret_cast<const uint4*>(row + k);
    if (row && k + 16 < K) v = *reinterpret_cast<const uint4*>(row + k + 16);
    return i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
}

__device__ __forceinline__ void store_y(const BlockGemmParams& p, int64_t row, int64_t col, float v) {
    if (p.y_bf16) reinterpret_cast<__bf16*>(p.y)[row * p.ldy + col] = (__bf16)v;
    else reinterpret_cast<float*>(p.y)[row * p.ldy + col] = v;
}

}  // namespace

// 64 x 64 tile, four wavefronts of 32 x 32; fragments straight from memory.
template <int FW, int FA>
__global__ void __launch_bounds__(256) block_gemm_direct_kernel(BlockGemmParams p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r32 = lane & 31, hk = lane >> 5;
    const int64_t e = p.experts ? blockIdx.z : 0;
    int64_t lo = 0, hi = p.M;
    if (p.experts) {
        lo = p.offsets[e] < 0 ? 0 : p.offsets[e];
        hi = p.offsets[e + 1] > p.M ? p.M : p.offsets[e + 1];
    }
    const int64_t n0 = (int64_t)blockIdx.x * 64 + (wave & 1) * 32;
    const uint8_t* w = p.w + e * p.stride_w;
    const float* ws = p.w_scales + e * p.stride_ws;
    for (int64_t m0 = lo + (int64_t)blockIdx.y * 64 + (wave >> 1) * 32; m0 < hi; m0 += (int64_t)gridDim.y * 64) {
        const int64_t m = m0 + r32, n = n0 + r32;
        int64_t out = m, src = m;
        if (m >= hi) {
            out = -1;
        } else if (p.experts) {
            out = p.slot_list[m];
            if (out < 0 || out >= p.M) out = -1;
            src = out / p.slots_per_row;
        }
        const uint8_t* arow = out >= 0 ? p.a + src * p.lda : nullptr;
        const uint8_t* wrow = n < p.N ? w + n * p.ldw : nullptr;
        f32x16 t = {};
        for (int64_t k = 0; k < p.K; k += 128) {
            f32x16 c = {};
            c = mfma64<FW, FA>(load32(wrow, k + 32 * hk, p.K), load32(arow, k + 32 * hk, p.K), c);
            c = mfma64<FW, FA>(load32(wrow, k + 64 + 32 * hk, p.K), load32(arow, k + 64 + 32 * hk, p.K), c);
            const float s = out >= 0 && n0 < p.N ? p.a_scales[src * p.lda_s + k / 128] * ws[n0 / 128 * p.ldw_s + k / 128] : 0.0f;
#pragma unroll
            for (int v = 0; v < 16; v++) t[v] = __builtin_fmaf(c[v], s, t[v]);
        }
        if (out >= 0) {
#pragma unroll
            for (int v = 0; v < 16; v++) {
                const int64_t col = n0 + 8 * (v / 4) + 4 * hk + v % 4;
                if (col < p.N) store_y(p, out, col, t[v]);
            }
        }
    }
}

template <int FW, int FA>
static hipError_t launch_direct(const BlockGemmParams& p, hipStream_t s) {
    const int64_t tiles = (p.M + 63) / 64;
    const dim3 grid((unsigned)((p.N + 63) / 64), (unsigned)(tiles > 1024 ? 1024 : tiles), (unsigned)(p.experts ? p.experts : 1));
    block_gemm_direct_kernel<FW, FA><<<grid, 256, 0, s>>>(p);
    return hipGetLastError();
}

hipError_t launch_gemm_block(const BlockGemmParams& p, hipStream_t s) {
    if (p.fw == 0) return p.fa == 0 ? launch_direct<0, 0>(p, s) : launch_direct<0, 1>(p, s);
    return p.fa == 0 ? launch_direct<1, 0>(p, s) : launch_direct<1, 1>(p, s);
}

}  // namespace fp4
