// Drives the host layer of the key/value cache (cache_api.cpp) under AddressSanitizer and
// UndefinedBehaviorSanitizer, on the CPU: launchers are stubs that check what reaches them,
// descriptors take sizes, strides, types and pointers from lists that hold the extremes.
// Device pointers are fake; the host layer must never dereference them.
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "../../include/fp4_cache.h"
#include "../../bit_floating_point_amd/csrc/cache_internal.h"

static long g_launches = 0;
extern "C" const char* hipGetErrorString(hipError_t) { return "stub"; }

static void need(bool ok, const char* what) {
    if (!ok) {
        std::printf("a launch with %s\n", what);
        std::abort();
    }
}

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Every row's last byte in 128 bits: positive strides that clear each other in some order.
static void check_cache(const fp4::CacheParams& c) {
    need(c.k && c.v && c.k != c.v && aligned(c.k, 16) && aligned(c.v, 16), "bad rows");
    need(c.pages >= 1 && c.kv_heads >= 1 && c.kv_heads <= 65535 && c.page_log >= 4 && c.page_log <= 16, "bad sizes");
    need(c.head_dim == 64 || c.head_dim == 96 || c.head_dim == 128 || c.head_dim == 192 || c.head_dim == 256, "a bad row");
    need((c.store == fp4::kStoreBf16) == (c.scales == fp4::kScaleNone), "codes without scales");
    need(c.scales == fp4::kScaleNone || (c.k_scales && c.v_scales && aligned(c.k_scales, 16) && aligned(c.v_scales, 16)), "bad scales");
    need(c.stride_page >= 0 && c.stride_head >= 0 && c.stride_page % 16 == 0 && c.stride_head % 16 == 0 && c.stride_row % 16 == 0, "odd strides");
    const int bits = c.store == fp4::kStoreBf16 ? 16 : c.store == fp4::kStoreE2m1 ? 4 : 8;
    need(c.stride_row >= (uint32_t)(c.head_dim * bits / 8) && ((uint64_t)c.stride_row << c.page_log) <= 0x7fffffff, "rows that overlap or are far apart");
    const __int128 last = (__int128)(c.pages - 1) * c.stride_page + (__int128)(c.kv_heads - 1) * c.stride_head;
    need(last < ((__int128)1 << 62), "an offset above 2^62");
    need(c.pages == 1 || c.stride_page > 0, "pages on top of each other");
    need(c.kv_heads == 1 || c.stride_head > 0, "heads on top of each other");
}

namespace fp4 {
static hipError_t check_rows(const CacheRowsParams& p) {
    check_cache(p.c);
    need(p.tokens > 0 && p.positions && p.k_rows && p.v_rows, "no tokens");
    need(p.ldk >= (int64_t)p.c.kv_heads * p.c.head_dim && p.ldv >= (int64_t)p.c.kv_heads * p.c.head_dim, "short rows");
    need(p.capacity >= 0 && p.capacity <= 1 << 30 && (p.capacity == 0 || p.sequences == 0 || p.table), "no table");
    ++g_launches;
    return hipSuccess;
}
hipError_t launch_cache_write(const CacheRowsParams& p, hipStream_t) { return check_rows(p); }
hipError_t launch_cache_read(const CacheRowsParams& p, hipStream_t) {
    need(p.k_rows != p.v_rows, "one output");
    return check_rows(p);
}
hipError_t launch_attend(const AttendParams& p, hipStream_t) {
    check_cache(p.c);
    need(p.sequences > 0 && p.heads > 0 && p.heads <= 65536 && p.share * p.c.kv_heads == p.heads, "bad heads");
    need(p.q && p.y && p.lengths && aligned(p.q, 16) && aligned(p.y, 16), "no rows");
    need(p.ldq >= (int64_t)p.heads * p.c.head_dim && p.ldy >= (int64_t)p.heads * p.c.head_dim, "short rows");
    need(p.capacity >= 0 && p.capacity <= 1 << 30 && (p.capacity == 0 || p.table) && p.window >= 0, "bad lengths");
    need(p.scale_log2 - p.scale_log2 == 0.0f, "a scale that is not finite");
    need(p.splits >= 1 && p.splits <= kMostSplits && p.splits == 1 << p.split_log, "bad parts");
    need(p.splits == 1 || (p.part_o && p.part_ml && aligned(p.part_o, 16)), "no workspace");
    // the device's parts fit those of the host, for the longest sequence and some others
    for (const int32_t n : {p.capacity, p.capacity / 2, p.capacity / 3}) {
        const SplitRange r = split_range(n, p.window, p.split_log, p.least_log);
        need(r.used() <= p.splits && r.first >= 0 && r.count >= 0 && r.count <= p.capacity, "more parts than there is room for");
    }
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

static const int64_t kSizes[] = {0, 1, 3, 16, 300, 4096, 65536, 1 << 20, -1, 1ll << 30, 1ll << 31, 1ll << 40, INT64_MAX, INT64_MIN};
static const int64_t kStrides[] = {0, 64, 128, 256, 2048, 4096, 8192, 1 << 20, 1ll << 33, 130, -128, 1ll << 40, 1ll << 60, INT64_MAX, INT64_MAX - 15, INT64_MIN};
static const int32_t kSmall[] = {0, 1, 1, 2, 4, 8, 32, 64, 65535, 65536, -1, INT32_MAX, INT32_MIN};
static const int32_t kTypes[] = {FP4_F32, FP4_BF16, FP4_BF16, FP4_F16, FP4_PACKED, -3, 99};
static const int32_t kDims[] = {64, 96, 128, 192, 256, 80, 0, -64, INT32_MAX};
static const int32_t kPageSizes[] = {16, 32, 64, 256, 65536, 131072, 24, 0, -16, INT32_MIN};
static const float kScales[] = {0.0f, 1.0f, -1.0f, 1.9e38f, 2.5e38f, 3.4e38f, -3.0e38f, __builtin_inff(), -__builtin_inff(), __builtin_nanf("")};
static const uintptr_t kPointers[] = {0x10000, 0x20000, 0, 0x10008, 0x10004, 0x10001};

// mostly the value that makes a call valid
template <typename T, typename V>
static T odd(T usual, const V& list) { return next() % 8 ? usual : (T)pick(list); }
static void* ptr(uintptr_t usual = 0x10000) { return reinterpret_cast<void*>(next() % 10 ? usual : pick(kPointers)); }
static void* maybe() { return next() % 2 ? nullptr : ptr(); }

static fp4_kv_cache cache() {
    static const int em[][2] = {{4, 3}, {5, 2}, {2, 1}, {2, 1}, {2, 3}, {9, -4}};
    fp4_kv_cache c;
    std::memset(&c, 0, sizeof c);
    c.k = ptr(), c.v = ptr(0x20000), c.pages = odd((int64_t)8, kSizes), c.kv_heads = odd(2, kSmall);
    c.head_dim = odd(kDims[next() % 5], kDims), c.page_size = odd(16 << next() % 3, kPageSizes);
    const bool bf16 = next() % 4 == 0;
    c.type = odd((int32_t)(bf16 ? FP4_BF16 : FP4_PACKED), kTypes);
    const int64_t row = 512, order = (int64_t)(next() % 3), size = c.page_size > 0 ? c.page_size : 16;
    c.stride_row = order == 0 ? row : order == 1 ? 2 * row : 16 * row;
    c.stride_head = order == 0 ? row * size : order == 1 ? row : 8 * row;
    c.stride_page = order == 2 ? row : 2 * row * size;
    c.stride_row = odd(c.stride_row, kStrides), c.stride_head = odd(c.stride_head, kStrides), c.stride_page = odd(c.stride_page, kStrides);
    const int* q = em[next() % 8 ? next() % 4 : next() % 6];
    if (!bf16) {
        c.grid.kind = next() % 20 ? FP4_GRID_MINIFLOAT : (int)(next() % 5);
        c.grid.e = q[0];
        c.grid.m = q[1];
        c.gran.mode = odd((int32_t)(next() % 2), kSmall);
        c.gran.scale_dtype = odd((int32_t)(c.gran.mode == FP4_SCALE_ROW && next() % 2 ? FP4_F16 : FP4_F32), kTypes);
        c.gran.group = odd(0, kSmall), c.gran.reserved = odd(0, kSmall);
        c.k_scales = ptr(), c.v_scales = ptr();
    } else if (next() % 16 == 0) {
        c.k_scales = ptr();
    }
    return c;
}

int main() {
    long ok = 0, refused = 0;
    auto count = [&](fp4_status s) {
        if (s == FP4_OK) ok++;
        else refused++;
        if (std::strlen(fp4_last_error()) > 511 || (s != FP4_OK && !fp4_last_error()[0])) std::abort();
    };
    for (long it = 0; it < 1000000; it++) {
        const fp4_kv_cache c = cache();
        {
            fp4_cache_rows_desc d;
            std::memset(&d, 0, sizeof d);
            d.page_table = (int32_t*)ptr(), d.sequences = odd((int64_t)4, kSizes), d.max_pages = odd((int64_t)64, kSizes);
            d.ld_table = odd((int64_t)64, kSizes), d.tokens = odd((int64_t)9, kSizes), d.positions = (int32_t*)ptr();
            d.sequence_of = (int32_t*)maybe(), d.k = ptr(), d.ldk = odd((int64_t)512, kStrides), d.v = ptr(0x20000);
            d.ldv = odd((int64_t)512, kStrides), d.dtype = odd((int32_t)FP4_BF16, kTypes), d.reserved = odd(0, kSmall);
            count(next() % 2 ? fp4_cache_write(&c, &d, nullptr) : fp4_cache_read(&c, &d, nullptr));
        }
        {
            fp4_attend_desc d;
            std::memset(&d, 0, sizeof d);
            d.sequences = odd((int64_t)4, kSizes), d.heads = odd(c.kv_heads > 0 && c.kv_heads < 9 ? 2 * c.kv_heads : 4, kSmall);
            d.q_dtype = odd((int32_t)FP4_F32, kTypes), d.q = ptr(), d.ldq = odd((int64_t)4096, kStrides), d.page_table = (int32_t*)ptr();
            d.max_pages = odd((int64_t)4096, kSizes), d.ld_table = odd((int64_t)4096, kSizes), d.lengths = (int32_t*)ptr();
            d.max_length = odd((int64_t)1 << 20, kSizes), d.window = odd((int64_t)0, kSizes), d.scale = odd(0.1f, kScales);
            d.y_dtype = odd((int32_t)FP4_BF16, kTypes), d.y = ptr(0x20000), d.ldy = odd((int64_t)4096, kStrides), d.lse = (float*)maybe();
            const size_t size = fp4_attend_workspace_size(d.sequences, d.heads, c.kv_heads, c.head_dim, d.max_length, d.window);
            count(fp4_attend(&c, &d, ptr(), next() % 8 ? size : (size_t)(next() % 4096), nullptr));
        }
        (void)fp4_attend_workspace_size(pick(kSizes), pick(kSmall), pick(kSmall), pick(kDims), pick(kSizes), pick(kSizes));
    }
    count(fp4_cache_write(nullptr, nullptr, nullptr));
    count(fp4_cache_read(nullptr, nullptr, nullptr));
    count(fp4_attend(nullptr, nullptr, nullptr, 0, nullptr));
    std::printf("%ld calls accepted, %ld refused, %ld launches\n", ok, refused, g_launches);
    return ok < 10000 || refused < 10000 || g_launches < 10000;
}
