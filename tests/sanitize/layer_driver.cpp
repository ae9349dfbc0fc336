// Drives the host layer of the layer operators (layer_api.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer, on the CPU: launchers are stubs that check what reaches them,
// descriptors take sizes, strides, types and pointers from lists that hold the extremes.
// Device pointers are fake; the host layer must never dereference them.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/fp4_layer.h"
#include "../../bit_floating_point_amd/csrc/layer_internal.h"

static long g_launches = 0;
extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

static void need(bool ok, const char* what) {
    if (!ok) {
        std::printf("a launch with %s\n", what);
        std::abort();
    }
}

namespace fp4 {
hipError_t launch_rmsnorm_quant(const NormParams& p, hipStream_t) {
    need(p.rows > 0 && p.cols > 0 && p.cols <= 65536 && p.cols % 8 == 0 && p.x && p.gamma && p.terms >= 1, "a bad norm");
    need(p.ldx >= p.cols && (!p.out.packed || p.out.ldp >= p.cols), "short rows");
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_swiglu_quant(const SwigluParams& p, hipStream_t) {
    need(p.rows > 0 && p.cols > 0 && p.cols <= 65536 && p.x && p.out.packed && p.ldx >= 2 * p.cols, "a bad SwiGLU");
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_quantize_block(const BlockQuantParams& p, hipStream_t) {
    need(p.batch > 0 && p.n > 0 && p.k > 0 && p.w && p.packed && p.scales, "bad blocks");
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_gemm_block(const BlockGemmParams& p, hipStream_t) {
    need(p.M > 0 && p.N > 0 && p.K > 0 && p.K % 16 == 0 && p.lda >= p.K && p.ldw >= p.K && p.a && p.w && p.y, "a bad product");
    need(p.lda < (1 << 22) && p.ldw < (1 << 22) && p.slots_per_row >= 1, "long rows");
    ++g_launches;
    return hipSuccess;
}
size_t route_workspace_bytes(int64_t tokens, int32_t experts, int32_t) { return (size_t)tokens * 4 + (size_t)experts; }
hipError_t launch_route(const RouteParams& p, hipStream_t) {
    need(p.tokens >= 0 && p.experts >= 1 && p.experts <= 1024 && p.top_k >= 1 && p.top_k <= 32 && p.top_k <= p.experts, "a bad routing");
    need(p.tokens == 0 || (p.logits && p.experts_out && p.weights_out), "null pointers");
    ++g_launches;
    return hipSuccess;
}
}  // namespace fp4

static uint64_t g_seed = 88172645463325252ull;
static uint64_t next() {
    g_seed ^= g_seed << 13;
    g_seed ^= g_seed >> 7;
    return g_seed ^= g_seed << 17;
}
template <typename T, size_t N>
static T pick(const T (&v)[N]) { return v[next() % N]; }

static const int64_t kSizes[] = {0, 1, 8, 16, 64, 128, 256, 256, 256, 4096, 65536, 100, -1, 1ll << 31, 1ll << 40, INT64_MAX, INT64_MIN};
static const int64_t kStrides[] = {0, 256, 512, 512, 4096, 1 << 20, 1 << 22, 260, -16, 1ll << 40, INT64_MAX, INT64_MAX - 15, INT64_MIN};
static const int32_t kSmall[] = {0, 1, 1, 1, 2, 4, 8, 32, 64, -1, 2000, INT32_MAX, INT32_MIN};
static const int32_t kTypes[] = {FP4_F32, FP4_BF16, FP4_BF16, FP4_F16, FP4_PACKED, -3, 99};
static const uintptr_t kPointers[] = {0x10000, 0x10000, 0x10000, 0x10000, 0x20000, 0, 0x10004, 0x10001};

// mostly the value that makes a call valid
template <typename T, typename V>
static T odd(T usual, const V& list) { return next() % 6 ? usual : (T)pick(list); }
static void* ptr() { return reinterpret_cast<void*>(next() % 6 ? (uintptr_t)0x10000 : pick(kPointers)); }
static void* maybe() { return next() % 2 ? nullptr : ptr(); }

static fp4_grid grid() {
    static const int em[][2] = {{4, 3}, {4, 3}, {5, 2}, {2, 1}, {2, 3}, {9, -4}};
    fp4_grid g;
    std::memset(&g, 0, sizeof g);
    const int* q = em[next() % 6];
    g.kind = next() % 10 ? FP4_GRID_MINIFLOAT : (int)(next() % 5);
    g.e = q[0];
    g.m = q[1];
    return g;
}
static fp4_gran gran() {
    static const int32_t groups[] = {0, 8, 64, 128, 512, 24, -8, INT32_MIN};
    fp4_gran g;
    std::memset(&g, 0, sizeof g);
    g.mode = odd(1 + (int32_t)(next() % 2), kSmall);
    g.group = g.mode == 2 ? odd(128, groups) : 0;
    g.scale_dtype = odd((int32_t)FP4_F32, kTypes);
    return g;
}

int main() {
    long ok = 0, refused = 0;
    auto count = [&](fp4_status s) {
        if (s == FP4_OK) ok++;
        else refused++;
        if (std::strlen(fp4_last_error()) > 511 || (s != FP4_OK && !fp4_last_error()[0])) std::abort();
    };
    for (long it = 0; it < 400000; it++) {
        {
            fp4_rmsnorm_desc d;
            std::memset(&d, 0, sizeof d);
            d.rows = odd((int64_t)4, kSizes), d.cols = odd((int64_t)256, kSizes), d.x = ptr(), d.ldx = odd((int64_t)512, kStrides);
            d.x_dtype = odd((int32_t)FP4_BF16, kTypes), d.terms = odd(1, kSmall), d.term_weights = (float*)maybe();
            d.residual = maybe(), d.ldr = odd((int64_t)512, kStrides), d.residual_out = maybe(), d.ldro = odd((int64_t)512, kStrides);
            d.residual_dtype = odd((int32_t)FP4_F32, kTypes), d.gamma_dtype = odd((int32_t)FP4_F32, kTypes), d.gamma = ptr();
            d.eps = 1e-6f, d.y_dtype = odd((int32_t)FP4_BF16, kTypes), d.y = maybe(), d.ldy = odd((int64_t)512, kStrides);
            d.grid = grid(), d.gran = gran(), d.tensor_scale = next() % 8 ? nullptr : (float*)ptr();
            d.packed = (uint8_t*)ptr(), d.ldp = odd((int64_t)512, kStrides), d.scales = ptr();
            count(fp4_rmsnorm_quant(&d, nullptr));
        }
        {
            fp4_swiglu8_desc d;
            std::memset(&d, 0, sizeof d);
            d.rows = odd((int64_t)4, kSizes), d.cols = odd((int64_t)256, kSizes), d.x = ptr(), d.ldx = odd((int64_t)512, kStrides);
            d.x_dtype = odd((int32_t)FP4_BF16, kTypes), d.grid = grid(), d.gran = gran();
            d.packed = (uint8_t*)ptr(), d.ldp = odd((int64_t)512, kStrides), d.scales = ptr();
            count(fp4_swiglu_quant(&d, nullptr));
        }
        count(fp4_quantize_block(ptr(), odd((int32_t)FP4_F32, kTypes), odd((int64_t)2, kSizes), odd((int64_t)64, kSizes),
                                 odd((int64_t)256, kSizes), odd((int64_t)512, kStrides), odd((int64_t)4096, kStrides), grid(),
                                 (uint8_t*)ptr(), odd((int64_t)512, kStrides), odd((int64_t)4096, kStrides), (float*)ptr(), nullptr));
        {
            fp4_gemm_block_desc d;
            std::memset(&d, 0, sizeof d);
            d.M = odd((int64_t)4, kSizes), d.N = odd((int64_t)64, kSizes), d.K = odd((int64_t)256, kSizes);
            d.a = (uint8_t*)ptr(), d.lda = odd((int64_t)512, kStrides), d.a_scales = (float*)ptr(), d.lda_s = odd((int64_t)512, kStrides);
            d.a_grid = grid(), d.w = (uint8_t*)ptr(), d.ldw = odd((int64_t)512, kStrides), d.w_scales = (float*)ptr();
            d.ldw_s = odd((int64_t)512, kStrides), d.w_grid = grid(), d.y = ptr(), d.ldy = odd((int64_t)512, kStrides);
            d.y_dtype = odd((int32_t)FP4_BF16, kTypes);
            count(fp4_gemm_block(&d, nullptr));
        }
        {
            fp4_route_desc d;
            std::memset(&d, 0, sizeof d);
            d.tokens = odd((int64_t)64, kSizes), d.experts = odd(64, kSmall), d.top_k = odd(4, kSmall), d.logits = ptr();
            d.ld = odd((int64_t)512, kStrides), d.logits_dtype = odd((int32_t)FP4_F32, kTypes), d.score = odd(0, kSmall);
            d.bias = (float*)maybe(), d.groups = odd(1, kSmall), d.top_groups = odd(1, kSmall), d.group_top = odd(1, kSmall);
            d.renormalise = pick(kSmall), d.scale = 1.0f, d.experts_out = (int32_t*)ptr(), d.weights_out = (float*)ptr();
            d.offsets = (int32_t*)ptr(), d.slots = (int32_t*)ptr();
            const size_t ws = next() % 4 ? (size_t)1 << 40 : (size_t)next() % 4096;
            count(fp4_route(&d, ptr(), ws, nullptr));
            (void)fp4_route_workspace_size(pick(kSizes), pick(kSmall), pick(kSmall));
        }
        {
            fp4_gemm_experts_desc d;
            std::memset(&d, 0, sizeof d);
            d.slots = odd((int64_t)64, kSizes), d.N = odd((int64_t)64, kSizes), d.K = odd((int64_t)256, kSizes);
            d.experts = odd(8, kSmall), d.slots_per_row = odd(4, kSmall), d.a = (uint8_t*)ptr(), d.lda = odd((int64_t)512, kStrides);
            d.a_scales = (float*)ptr(), d.lda_s = odd((int64_t)512, kStrides), d.a_grid = grid(), d.w = (uint8_t*)ptr();
            d.ldw = odd((int64_t)512, kStrides), d.stride_w = odd((int64_t)32768, kStrides), d.w_scales = (float*)ptr();
            d.w_grid = grid(), d.offsets = (int32_t*)ptr(), d.slot_list = (int32_t*)ptr(), d.y = ptr();
            d.ldy = odd((int64_t)512, kStrides), d.y_dtype = odd((int32_t)FP4_BF16, kTypes);
            count(fp4_gemm_experts(&d, nullptr));
        }
    }
    count(fp4_rmsnorm_quant(nullptr, nullptr));
    count(fp4_swiglu_quant(nullptr, nullptr));
    count(fp4_gemm_block(nullptr, nullptr));
    count(fp4_route(nullptr, nullptr, 0, nullptr));
    count(fp4_gemm_experts(nullptr, nullptr));
    if (ok < 1000 || refused < 1000 || g_launches < 1000) return 1;
    std::printf("%ld calls accepted, %ld refused, %ld launches\n", ok, refused, g_launches);
    return 0;
}
