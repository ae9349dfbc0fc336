// Internal declarations of the layer operators (include/fp4_layer.h): parameters that the
// host layer (layer_api.cpp) passes to the HIP kernels, and the helpers of fp4_api.cpp
// that both host files use.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp4.h"
#include "fp4_internal.h"

namespace fp4 {

// fp4_api.cpp: the calling thread's error message with a status; a grid's table; the
// checks of a granularity that do not involve a row length
fp4_status report(fp4_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fp4_status report_ok();
fp4_status report_hip(hipError_t e, const char* what);
fp4_status grid_table(const fp4_grid& g, QGrid* q);

constexpr int kBlock = 128;  // rows and columns of a scale block

// Workgroups of one launch: its threads number less than 2^32.  Past that the grid wraps and the
// rest does not run, with no error, so launchers split larger work.
inline int64_t max_workgroups(int threads) { return 0xffffffffll / threads; }

// where 8-bit codes and their scales go
struct CodeOut {
    uint8_t* packed;  // null: no codes
    int64_t ldp;      // bytes
    int32_t e4m3;     // else E5M2
    int32_t mode;     // 0 tensor (scale given), 1 row, 2 group
    int32_t group;
    int32_t scale_f16;
    float qmax, rqmax;  // largest magnitude and fl32 of one over it
    const float* tensor_scale;
    const int8_t* col_shift;
    void* scales;
};

struct NormParams {
    int64_t rows, cols;
    const void* x;
    int64_t ldx;
    int32_t x_bf16;
    int32_t terms;
    const float* term_weights;
    const void* residual;
    int64_t ldr;
    void* residual_out;
    int64_t ldro;
    int32_t residual_bf16;
    int32_t gamma_bf16;
    const void* gamma;
    float eps;
    int32_t y_bf16;
    void* y;
    int64_t ldy;
    CodeOut out;
};
hipError_t launch_rmsnorm_quant(const NormParams& p, hipStream_t s);

struct SwigluParams {
    int64_t rows, cols;
    const void* x;
    int64_t ldx;
    int32_t x_bf16;
    CodeOut out;
};
hipError_t launch_swiglu_quant(const SwigluParams& p, hipStream_t s);

struct BlockQuantParams {
    const void* w;
    int32_t bf16;
    int64_t batch, n, k, ldw, stride_w;
    int32_t e4m3;
    float qmax;
    uint8_t* packed;
    int64_t ldp, stride_p;
    float* scales;
};
hipError_t launch_quantize_block(const BlockQuantParams& p, hipStream_t s);

// Y = X W^T with block scales; experts > 0: the experts' products (M = slots)
struct BlockGemmParams {
    int64_t M, N, K;
    const uint8_t* a;
    int64_t lda;
    const float* a_scales;
    int64_t lda_s;
    const uint8_t* w;
    int64_t ldw, stride_w;
    const float* w_scales;
    int64_t ldw_s, stride_ws;  // elements; stride_ws between experts
    void* y;
    int64_t ldy;
    int32_t y_bf16;
    int32_t fa, fw;  // matrix-core format codes: 0 E4M3, 1 E5M2
    int32_t experts;
    int32_t slots_per_row;
    const int32_t* offsets;
    const int32_t* slot_list;
};
hipError_t launch_gemm_block(const BlockGemmParams& p, hipStream_t s);

struct RouteParams {
    int64_t tokens;
    int32_t experts, top_k;
    const void* logits;
    int64_t ld;
    int32_t logits_bf16;
    int32_t sigmoid;
    const float* bias;
    int32_t groups, top_groups, group_top;
    int32_t renormalise;
    float scale;
    int32_t* experts_out;
    float* weights_out;
    int32_t* offsets;
    int32_t* slots;
    int32_t* counts;  // workspace
};
size_t route_workspace_bytes(int64_t tokens, int32_t experts, int32_t top_k);
hipError_t launch_route(const RouteParams& p, hipStream_t s);

}  // namespace fp4
