// Attention of one new token per sequence over the pages of a cache: the kernel over a part
// of a sequence.  Instances: attend_bf16.hip, attend_e4m3.hip, attend_e5m2.hip, attend_e2m1.hip.
//
// Mathematics.  One pass: m the largest z seen so far (any upper estimate to 2^8 will do), l = sum of
// 2^(z - m), O = sum of 2^(z - m) V; a larger z scales l and O by 2^(m - m').  Parts (m, l, O)
// are joined with factors 2^(m_i - M).  z is in powers of two: the scale holds log2 e.
//
// Layout.  A wavefront takes 32 positions at a time, as two halves of 16 (a page holds a multiple of 16
// positions, so a half lies in one page and has a base address of its own), with the 16x16x32
// bf16 matrix instruction, whose operands a lane holds as 8 values along the summed dimension:
//   Z^T = K Q^T: rows are 16 positions, columns 16 query heads, summed over 32 columns of K;
//   O^T = V^T P^T: rows are 16 columns of V, columns the heads, summed over the 32 positions.
// Lane (n = lane % 16, g = lane / 16) gets Z of head n and positions 4g .. 4g + 3 of both halves; the
// positions' order along the sum over P is free, so those 8 numbers ARE the lane's operand
// of the second product.  Maxima, sums and factors of head n stay in its lanes.
//   K: lane (n, g) reads row n, g's pieces of it, as they are needed (the order of columns along
//      the sum is free too: q is read in the same order).
//   V: lane (n, g) reads the same few columns of its 8 positions, 16 lanes a whole row; pairs of positions
//      are interleaved by byte permutes and converted two at a time.
// Codes convert to bf16 exactly, scales of rows go into z and into the weights p = 2^(z - m), which are sums of
// two or three bf16 terms: one would be off by 2^-9.
//
// Bounds.  Rows of 8 bits and more: reading the cache.  16 sequences of 4096 positions, 40 heads of 128, E4M3: 114 us, 6.1 TB/s; one of
// 131072, 8 kv heads of 128, bf16: 86 us, 6.3 TB/s, a streaming read's rate.  E2M1 converts twice as many values a byte: 96
// sequences of up to 8192 positions, 8 kv heads with 8 heads each, 92 us, 4.6 TB/s; vector instructions (215 a tile)
// take 43% of the SIMDs' cycles and matrix instructions 18%, waiting for loads and the ragged end the rest.
// Scales converted where they are used, scalar bases, no load that anything waits for but its use: 175 -> 92.
#pragma once
#include <type_traits>

#include "cache_internal.h"
#include "unit_codes.h"

namespace fp4 {

namespace attend {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = kAttendWaves * 64;
constexpr float kNothing = -3.0e38f;  // z of a position that is not seen; m before the first
constexpr float kSlack = 8.0f;        // log2 of the largest weight: z may pass m by this much

// `total` things in pieces of powers of two, none above `most`: number, start and size
constexpr int piece_size(int total, int most, int l) {
    int at = 0, size = 0;
    for (int i = 0; i <= l; i++) {
        at += size;
        size = 1;
        while (2 * size <= most && 2 * size <= total - at) size *= 2;
    }
    return size;
}
constexpr int piece_first(int total, int most, int l) {
    int at = 0;
    for (int i = 0; i < l; i++) at += piece_size(total, most, i);
    return at;
}
constexpr int pieces(int total, int most) {
    int n = 0;
    while (piece_first(total, most, n) < total) n++;
    return n;
}

// What a lane loads of a tile.  K: D / 32 steps of 8 columns a lane, in loads of up to 16 bytes.
// V: D / 16 columns a lane, likewise.
template <int STORE, int D>
struct Plan {
    static constexpr int kBits = STORE == kStoreBf16 ? 16 : STORE == kStoreE2m1 ? 4 : 8;
    static constexpr int kSteps = D / 32, kStepBytes = kBits;  // bytes of 8 columns
    static constexpr int kLoads = pieces(kSteps, 16 / kStepBytes);
    static constexpr int k_first(int l) { return piece_first(kSteps, 16 / kStepBytes, l); }
    static constexpr int k_steps(int l) { return piece_size(kSteps, 16 / kStepBytes, l); }
    static constexpr int kCols = D / 16;
    static constexpr int vLoads = pieces(kCols, 128 / kBits);
    static constexpr int v_first(int l) { return piece_first(kCols, 128 / kBits, l); }
    static constexpr int v_cols(int l) { return piece_size(kCols, 128 / kBits, l); }
    static constexpr int v_bytes(int l) { return v_cols(l) * kBits / 8; }
    static constexpr int v_words(int l) { return (v_bytes(l) + 3) / 4; }
    static constexpr int v_word_first(int l) { return l == 0 ? 0 : v_word_first(l - 1) + v_words(l - 1); }
    static constexpr int kWords = kSteps * kStepBytes / 4, vWords = v_word_first(vLoads);
};

// BYTES of a lane at byte `off` + `more` (one of all lanes) past a buffer's start.  Buffer loads: base
// and `more` are scalars, so a load costs no vector instruction for its address.
constexpr int kOnce = 2;  // nontemporal
template <int BYTES>
__device__ __forceinline__ void load_bytes(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t more, uint32_t* w) {
    if constexpr (BYTES == 16) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off, more, kOnce);
        w[0] = v[0], w[1] = v[1], w[2] = v[2], w[3] = v[3];
    } else if constexpr (BYTES == 8) {
        const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, off, more, kOnce);
        w[0] = v[0], w[1] = v[1];
    } else if constexpr (BYTES == 4) {
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(r, off, more, kOnce);
    } else if constexpr (BYTES == 2) {
        w[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, off, more, kOnce);
    } else {
        w[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(r, off, more, kOnce);
    }
}
// The buffer from `base` + off on: pages and scales are addressed by their own starts, offsets stay below
// 2^31.  With `there` false it is empty: loads give zeros and read nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* base, int64_t off, bool there) {
    return buf_make(reinterpret_cast<const uint8_t*>(base) + off, there ? 0x7fffffff : 0);
}

__device__ __forceinline__ uint32_t bits(bf16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ bf16x8 operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}

// two codes of a word as bf16: those in half `HALF` (8 bits) or byte `AT` (4 bits)
template <int STORE, int AT>
__device__ __forceinline__ uint32_t two_values(uint32_t w) {
    if constexpr (STORE == kStoreE4m3) return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, AT != 0));
    else if constexpr (STORE == kStoreE5m2) return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, AT != 0));
    else return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, AT));
}

// 8 columns of a row of K, from the words at w
template <int STORE>
__device__ __forceinline__ bf16x8 key_operand(const uint32_t* w) {
    if constexpr (STORE == kStoreBf16) {
        return operand(w[0], w[1], w[2], w[3]);
    } else if constexpr (STORE == kStoreE2m1) {
        return operand(two_values<STORE, 0>(w[0]), two_values<STORE, 1>(w[0]), two_values<STORE, 2>(w[0]), two_values<STORE, 3>(w[0]));
    } else {
        return operand(two_values<STORE, 0>(w[0]), two_values<STORE, 1>(w[0]), two_values<STORE, 0>(w[1]), two_values<STORE, 1>(w[1]));
    }
}

// Column E of the word w[.] of 8 positions: pairs of positions side by side.  The interleaved
// words serve 2 (bf16), 4 (8 bits) or 8 (4 bits) columns; the compiler keeps them.
template <int STORE, int E>
__device__ __forceinline__ uint32_t value_pair(uint32_t a, uint32_t b) {
    if constexpr (STORE == kStoreBf16) {
        return __builtin_amdgcn_perm(b, a, E == 0 ? 0x05040100u : 0x07060302u);
    } else if constexpr (STORE == kStoreE2m1) {
        constexpr uint32_t low = 0x0f0f0f0fu;
        const uint32_t w = E % 2 == 0 ? (a & low) | ((b << 4) & ~low) : ((a >> 4) & low) | (b & ~low);
        return two_values<STORE, E / 2>(w);
    } else {
        return two_values<STORE, E % 2>(__builtin_amdgcn_perm(b, a, E < 2 ? 0x05010400u : 0x07030602u));
    }
}

__device__ __forceinline__ float low_half(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_half(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// x (8 values) as sums of N bf16 terms, each the nearest to what is left
template <int N>
__device__ __forceinline__ void terms_of(float x[8], bf16x8 out[N]) {
#pragma unroll
    for (int t = 0; t < N; t++) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            w[i] = bf16_pair(x[2 * i], x[2 * i + 1]);
            asm("" : "+v"(w[i]));  // the pair is at hand: its halves are not converted again
            x[2 * i] -= low_half(w[i]);
            x[2 * i + 1] -= high_half(w[i]);
        }
        out[t] = operand(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ float power2(float x) { return __builtin_amdgcn_exp2f(x); }

// the logarithm of a sum of exponentials: 2^m times `sum`
__device__ __forceinline__ float log_sum(float m, float sum) { return sum == 0.0f ? -INFINITY : (m + log2f(sum)) * 0x1.62e43p-1f; }

// four values into a row of f32 or bf16
__device__ __forceinline__ void put4(void* base, bool bf16, int64_t at, const f32x4& v) {
    if (bf16) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(base) + at) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    else *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(base) + at) = v;
}

// v is used here, so that its load is waited for here
__device__ __forceinline__ void arrived(bf16x8& v) { asm volatile("" : "+v"(v)); }

// f(integral_constant<0>) .. f(integral_constant<N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void repeat(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        repeat<N, I + 1>(f);
    }
}

// Row scales of a tile: a lane's four of each half, as they are stored until they are used.
// SCALES: kScaleRowF32, kScaleRowF16, or kScaleNone where there are none (one given scale is the
// caller's factor).
template <int SCALES>
struct RowScales {
    static constexpr int kBytes = SCALES == kScaleRowF32 ? 4 : SCALES == kScaleRowF16 ? 2 : 0;
    uint32_t w[2][4];
    // `first`: index of the half's first scale
    __device__ __forceinline__ void load(const void* scales, int64_t first, int half, int g, bool there) {
        if constexpr (kBytes) load_bytes<4 * kBytes>(buffer_at(scales, first * kBytes, there), (uint32_t)(4 * g * kBytes), 0, w[half]);
    }
    // x * (row j's scale) + y, rounded once: one instruction, binary16 scales are converted inside it
    __device__ __forceinline__ float fma(int j, float x, float y) const {
        const uint32_t* h = w[j / 4];
        if constexpr (SCALES == kScaleRowF32) return __builtin_fmaf(x, __uint_as_float(h[j % 4]), y);
        else return __builtin_fmaf(x, (float)__builtin_bit_cast(_Float16, (uint16_t)(h[j % 4 / 2] >> (16 * (j % 2)))), y);
    }
};

// Wavefronts per SIMD that a kernel has registers for, at least.  Two: with no more than 256
// registers the matrix instructions keep their sums in ordinary ones, where O is scaled in place
// (ragged E2M1 113 -> 101 us).  The widest rows do not fit those.
constexpr int least_waves(int store, int dim, bool wide) {
    const bool bf16 = store == kStoreBf16;
    return (dim == 256 && (bf16 || (wide && store != kStoreE2m1))) || (dim == 192 && bf16 && wide) ? 1 : 2;
}

// Whether a workgroup takes two tiles of query heads: keys and values are then read and converted once for
// 32 heads (one tile / two: 64 sequences of 8192, 64 heads on one, E4M3 112 / 65 us, bf16 185 / 103, E2M1 64 / 47;
// 16 of 4096, 20 heads on each of 3, E4M3 27 / 22).  Up to rows of 128 values and without the terms of f32
// there are registers for it.
constexpr bool two_tiles(int share, int dim, bool wide) { return share > kHeadTile && dim <= 128 && !wide; }

// WIDE: q or y is f32, and its terms three.  T: tiles of query heads of a workgroup.
template <int STORE, int SCALES, int D, bool WIDE, int T>
__global__ void __launch_bounds__(kThreads, least_waves(STORE, D, WIDE)) attend_kernel(AttendParams p, int64_t first_sequence) {
    using L = Plan<STORE, D>;
    constexpr int kHeads = T * kHeadTile;
    constexpr int kQTerms = WIDE ? 3 : 1, kPTerms = WIDE ? 3 : 2;
    constexpr int kRound = 8;  // heads whose parts are joined at a time
    constexpr int H = 2, J = 4 * H;  // halves of a tile, a lane's positions in it
    __shared__ float joined[kAttendWaves][kRound][D + 4];
    __shared__ float2 stats[kAttendWaves][kHeads];

    const CacheParams& c = p.c;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // Workgroup (kv head and tile of its query heads, sequence, part).  Workgroups go to the eight XCDs in turn:
    // with parts first, those that most sequences do not have would leave the same XCDs idle (33
    // sequences of 1000 positions: 17 against 9 us).
    const uint32_t tiles = (uint32_t)(p.share + kHeads - 1) / kHeads;
    const int split = (int)blockIdx.z, kv_head = (int)(tiles == 1 ? blockIdx.x : blockIdx.x / tiles);
    const int head_tile = (int)(blockIdx.x - (uint32_t)kv_head * tiles);
    const int64_t sequence = first_sequence + blockIdx.y;
    const int heads = min(p.share - head_tile * kHeads, kHeads);  // of this workgroup
    const int64_t first_head = (int64_t)kv_head * p.share + head_tile * kHeads;

    const int32_t length = __builtin_amdgcn_readfirstlane(max(0, min(p.lengths[sequence], p.capacity)));
    const SplitRange range = split_range(length, p.window, p.split_log, p.least_log);
    if (split > 0 && !range.has(split)) return;
    const int begin = range.first + split * range.chunk;
    const int end = length - begin < range.chunk ? length : begin + range.chunk;
    const int all = (end - begin + kTilePositions - 1) / kTilePositions;  // tiles of the part
    const int count = (all - wave + kAttendWaves - 1) / kAttendWaves;     // of this wavefront (at most 0: none)

    // z = dot * factor * (row's scale)
    constexpr bool kRows = SCALES != kScaleNone;
    float factor = p.scale_log2, v_all = 1.0f;
    if (c.scales == kScaleGiven) {
        factor *= *reinterpret_cast<const float*>(c.k_scales);
        v_all = *reinterpret_cast<const float*>(c.v_scales);
    }

    // q of heads n (, n + 16), in K's order of columns: loaded here, in terms once the first tile is on its way
    bf16x8 q[T][kQTerms][L::kSteps];
    Raw8 q_raw[T][WIDE ? L::kSteps : 1];
    const bool q_bf16 = !WIDE || p.q_bf16;
#pragma unroll
    for (int t = 0; t < T; t++) {
        const int64_t row = sequence * p.ldq + (first_head + t * kHeadTile + n) * D;
        repeat<L::kLoads>([&](auto x) {
            constexpr int first = L::k_first(x), steps = L::k_steps(x);
#pragma unroll
            for (int i = 0; i < steps; i++) {
                const int64_t col = row + first * 32 + g * 8 * steps + 8 * i;
                uint4 a{}, b{};
                if (t * kHeadTile + n < heads) {
                    if (q_bf16) {
                        a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(p.q) + col);
                    } else {
                        a = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p.q) + col)[0];
                        b = reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p.q) + col)[1];
                    }
                }
                if constexpr (WIDE) q_raw[t][first + i] = Raw8{a, b};
                else q[t][0][first + i] = __builtin_bit_cast(bf16x8, a);
            }
        });
    }

    float m[T] = {}, l[T] = {};
    bool fresh = true;  // nothing was seen yet
    f32x4 acc[T][L::kCols];
    repeat<T * L::kCols>([&](auto j) { acc[j / L::kCols][j % L::kCols] = f32x4{0.0f, 0.0f, 0.0f, 0.0f}; });

    uint32_t kw[H][L::kWords], vw[J][L::vWords];  // the tile on its way
    RowScales<SCALES> ks, vs;

    // Where the halves of the next 64 / H of this wavefront's tiles lie, one half a lane: the byte offset of
    // the first of the 16 rows and the index of its scale.  A half that is not in the cache or has nothing
    // to be seen: page 0 in its place, read and not used, and the highest bit set.
    const int32_t* table = p.table + sequence * p.ld_table;
    const int slots = (1 << c.page_log) - 1;
    constexpr uint32_t kAbsent = 0x80000000u;
    uint32_t row_low = 0, row_high = 0, scale_low = 0, scale_high = 0;
    auto find_pages = [&](int i) {
        const int t = begin + ((i + lane / H) * kAttendWaves + wave) * kTilePositions + 16 * (lane % H);
        const int found = t < end ? page_at(table + (t >> c.page_log), c.pages) : -1, page = max(found, 0);
        const int64_t row = page * c.stride_page + kv_head * c.stride_head + (int64_t)(t & slots) * c.stride_row;
        row_low = (uint32_t)row;
        row_high = (uint32_t)(row >> 32) | (found < 0 ? kAbsent : 0);
        if constexpr (kRows) {
            const int64_t scale = (((int64_t)page * c.kv_heads + kv_head) << c.page_log) + (t & slots);
            scale_low = (uint32_t)scale;
            scale_high = (uint32_t)(scale >> 32);
        }
    };
    // a tile of this wavefront: its first position, and where its halves lie
    struct Tile {
        int t;
        bool there;        // else past the last one, and nothing is loaded
        uint32_t high[H];  // kAbsent
        int64_t row[H], scale[H];
    };
    auto tile_of = [&](int i) {
        Tile r;
        r.t = begin + (i * kAttendWaves + wave) * kTilePositions;
        r.there = i < count;
#pragma unroll
        for (int h = 0; h < H; h++) {
            const int from = H * (i & (64 / H - 1)) + h;
            r.high[h] = __builtin_amdgcn_readlane(row_high, from);
            r.row[h] = (int64_t)(((uint64_t)(r.high[h] & ~kAbsent) << 32) | (uint32_t)__builtin_amdgcn_readlane(row_low, from));
            if constexpr (kRows)
                r.scale[h] = (int64_t)(((uint64_t)(uint32_t)__builtin_amdgcn_readlane(scale_high, from) << 32) |
                                       (uint32_t)__builtin_amdgcn_readlane(scale_low, from));
        }
        return r;
    };
    const uint32_t key_row = (uint32_t)n * c.stride_row, value_row = (uint32_t)(4 * g) * c.stride_row;
    auto load_keys = [&](const Tile& tile) {
#pragma unroll
        for (int h = 0; h < H; h++) {
            const auto rows = buffer_at(c.k, tile.row[h], tile.there);
            repeat<L::kLoads>([&](auto x) {
                constexpr int first = L::k_first(x), steps = L::k_steps(x), bytes = steps * L::kStepBytes;
                load_bytes<bytes>(rows, key_row + (uint32_t)(first * 4 * L::kStepBytes + g * bytes), 0, kw[h] + first * L::kStepBytes / 4);
            });
            ks.load(c.k_scales, tile.scale[h], h, g, tile.there);
        }
    };
    auto load_values = [&](const Tile& tile) {
#pragma unroll
        for (int h = 0; h < H; h++) {
            const auto rows = buffer_at(c.v, tile.row[h], tile.there);
#pragma unroll
            for (int j = 0; j < 4; j++)
                repeat<L::vLoads>([&](auto x) {
                    constexpr int bytes = L::v_bytes(x), first = L::v_first(x), word = L::v_word_first(x);
                    load_bytes<bytes>(rows, value_row + (uint32_t)(first * 2 * L::kBits + n * bytes), (uint32_t)j * c.stride_row,
                                      vw[4 * h + j] + word);
                });
            vs.load(c.v_scales, tile.scale[h], h, g, tile.there);
        }
    };

    Tile tile;
    // Tile i.  The loads of tile i + 1 start where the registers of i's keys and then of its values are free.
    // (Past the last tile they are of empty buffers: loads under a condition would be waited for where the
    // condition ends.)
    auto step = [&](int i) {
        // Z^T of every half
        f32x4 z[T][H];
#pragma unroll
        for (int h = 0; h < T * H; h++) z[h / H][h % H] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < L::kSteps; s++)
#pragma unroll
            for (int h = 0; h < H; h++) {
                const bf16x8 a = key_operand<STORE>(kw[h] + s * L::kStepBytes / 4);
#pragma unroll
                for (int t = 0; t < T; t++)
#pragma unroll
                    for (int k = kQTerms - 1; k >= 0; k--) z[t][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, q[t][k][s], z[t][h], 0, 0, 0);
            }
        // x = z - m
        float x[T][J];
#pragma unroll
        for (int t = 0; t < T; t++)
#pragma unroll
            for (int j = 0; j < J; j++) {
                const float dot = z[t][j / 4][j % 4];
                if constexpr (kRows) x[t][j] = ks.fma(j, dot * factor, -m[t]);
                else x[t][j] = __builtin_fmaf(dot, factor, -m[t]);
            }
        if (((i + 1) & (64 / H - 1)) == 0) find_pages(i + 1);
        const Tile next = tile_of(i + 1);
        load_keys(next);
        // What is not seen has no weight, whatever its rows and scales hold.  (It may call for a new
        // reference in vain.)
        uint32_t absent = 0;
        float most = x[0][0];
#pragma unroll
        for (int h = 0; h < H; h++) absent |= tile.high[h];
#pragma unroll
        for (int j = 1; j < T * J; j++) most = fmaxf(most, x[j / J][j % J]);
        const bool whole = tile.t >= range.begin && tile.t + kTilePositions <= end && (absent & kAbsent) == 0;
        auto seen = [&](int j) {
            const int t = tile.t + 16 * (j / 4) + 4 * g + j % 4;
            return whole | ((t >= range.begin) & (t < end) & ((tile.high[j / 4] & kAbsent) == 0));
        };
        if (fresh | __any(most > kSlack)) {
            const bool first = fresh;
#pragma unroll
            for (int t = 0; t < T; t++) {
                float top = kNothing;
#pragma unroll
                for (int j = 0; j < J; j++) top = fmaxf(top, seen(j) ? x[t][j] : kNothing);
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                // m moves to the first tile's largest z that has any (it was 0 until then), then upwards
                const bool none = __all(top <= kNothing);
                top = none ? 0.0f : first ? top : fmaxf(top, 0.0f);
                const float f = first ? 1.0f : power2(-top);
                fresh &= none;
                m[t] += top;
                l[t] *= f;
                repeat<L::kCols>([&](auto j) { acc[t][j] *= f; });
#pragma unroll
                for (int j = 0; j < J; j++) x[t][j] -= top;
            }
        }
#pragma unroll
        for (int j = 0; j < T * J; j++) x[j / J][j % J] = power2(x[j / J][j % J]);
        if (!whole) {
#pragma unroll
            for (int j = 0; j < T * J; j++) x[j / J][j % J] = seen(j % J) ? x[j / J][j % J] : 0.0f;
        }
#pragma unroll
        for (int t = 0; t < T; t++)
#pragma unroll
            for (int j = 0; j < J; j++) {
                l[t] += x[t][j];
                if constexpr (kRows) x[t][j] = vs.fma(j, x[t][j], 0.0f);
            }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < J; j++) {
                if constexpr (kRows) {
#pragma unroll
                    for (int t = 0; t < T; t++) x[t][j] = seen(j) ? x[t][j] : 0.0f;
                }
#pragma unroll
                for (int u = 0; u < L::vWords; u++) vw[j][u] = seen(j) ? vw[j][u] : 0u;
            }
        }
        bf16x8 weight[T][kPTerms];
#pragma unroll
        for (int t = 0; t < T; t++) terms_of<kPTerms>(x[t], weight[t]);
        // O^T: a column of V at a time
        repeat<L::vLoads>([&](auto y) {
            repeat<L::v_cols(y)>([&](auto e) {
                constexpr int per = 32 / L::kBits, word = L::v_word_first(y) + e / per, col = L::v_first(y) + e;
                const bf16x8 a = operand(value_pair<STORE, e % per>(vw[0][word], vw[1][word]), value_pair<STORE, e % per>(vw[2][word], vw[3][word]),
                                         value_pair<STORE, e % per>(vw[4][word], vw[5][word]), value_pair<STORE, e % per>(vw[6][word], vw[7][word]));
#pragma unroll
                for (int t = 0; t < T; t++) {
                    f32x4& o = acc[t][col];
#pragma unroll
                    for (int k = kPTerms - 1; k >= 0; k--) o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, weight[t][k], o, 0, 0, 0);
                }
            });
        });
        load_values(next);
        tile = next;
    };
    if (count > 0) {
        find_pages(0);
        tile = tile_of(0);
        load_keys(tile);
        load_values(tile);
        // q is waited for here, beside those: in the loop it would be waited for, with all loads, in every turn
#pragma unroll
        for (int t = 0; t < T; t++)
#pragma unroll
            for (int s = 0; s < L::kSteps; s++) {
                if constexpr (WIDE) {
                    float x[8];
                    if (q_bf16) raw8_to_float<true>(q_raw[t][s], x);
                    else raw8_to_float<false>(q_raw[t][s], x);
                    bf16x8 terms[kQTerms];
                    terms_of<kQTerms>(x, terms);
#pragma unroll
                    for (int k = 0; k < kQTerms; k++) q[t][k][s] = terms[k];
                }
                arrived(q[t][0][s]);
            }
        for (int i = 0; i < count; i++) step(i);
    }
    // The wavefronts' parts, joined: each scales its own O to the largest m (and over the sum, if this is the
    // only part), then they are added in order.  Lane (n, g) holds columns first * 16 + cols (4 g + i) + e.
#pragma unroll
    for (int t = 0; t < T; t++) {
        if (fresh) m[t] = kNothing;
        l[t] += __shfl_xor(l[t], 16, 64);
        l[t] += __shfl_xor(l[t], 32, 64);
        if (g == 0) stats[wave][t * kHeadTile + n] = make_float2(m[t], l[t]);
    }
    __syncthreads();
    const bool alone = range.count <= range.chunk;
    const int64_t head = sequence * p.heads + first_head;  // of n = 0
#pragma unroll
    for (int t = 0; t < T; t++) {
        const int at = t * kHeadTile + n;
        float top = stats[0][at].x, sum = 0.0f;
#pragma unroll
        for (int v = 1; v < kAttendWaves; v++) top = fmaxf(top, stats[v][at].x);
#pragma unroll
        for (int v = 0; v < kAttendWaves; v++) sum = __builtin_fmaf(stats[v][at].y, power2(stats[v][at].x - top), sum);
        float own = power2(m[t] - top) * v_all;
        if (alone) own *= sum == 0.0f ? 0.0f : 1.0f / sum;
        if (wave == 0 && g == 0 && at < heads) {
            if (!alone) *reinterpret_cast<float2*>(p.part_ml + ((head + at) * p.splits + split) * 2) = make_float2(top, sum);
            else if (p.lse) p.lse[head + at] = log_sum(top, sum);
        }
        const int last = min(heads, (t + 1) * kHeadTile);
        for (int r = t * kHeadTile; r < last; r += kRound) {
            if (r > 0) __syncthreads();
            if (at >= r && at < r + kRound) {
                repeat<L::vLoads>([&](auto x) {
                    repeat<L::v_cols(x)>([&](auto e) {
                        constexpr int cols = L::v_cols(x), first = L::v_first(x);
#pragma unroll
                        for (int i = 0; i < 4; i++) joined[wave][at - r][first * 16 + cols * (4 * g + i) + e] = acc[t][first + e][i] * own;
                    });
                });
            }
            __syncthreads();
            for (int e = threadIdx.x * 4; e < min(last - r, kRound) * D; e += kThreads * 4) {
                const int row = e / D, col = e % D;
                f32x4 o = *reinterpret_cast<const f32x4*>(&joined[0][row][col]);
#pragma unroll
                for (int v = 1; v < kAttendWaves; v++) o += *reinterpret_cast<const f32x4*>(&joined[v][row][col]);
                if (!alone) *reinterpret_cast<f32x4*>(p.part_o + ((head + r + row) * p.splits + split) * D + col) = o;
                else put4(p.y, p.y_bf16, sequence * p.ldy + (first_head + r + row) * D + col, o);
            }
        }
    }
}

// the kernel for the scales, the head dimension and the types of a call on one kind of cache
template <int STORE>
hipError_t launch_parts(const AttendParams& p, hipStream_t s) {
    const bool wide = !p.q_bf16 || !p.y_bf16;
    const int tiles = two_tiles(p.share, p.c.head_dim, wide) ? 2 : 1;
    const int64_t units = (int64_t)p.c.kv_heads * ((p.share + tiles * kHeadTile - 1) / (tiles * kHeadTile));
    int64_t most = max_workgroups(kThreads) / (units * p.splits);
    if (most > 65535) most = 65535;  // of a grid's second dimension
    for (int64_t first = 0; first < p.sequences; first += most) {
        const int64_t n = p.sequences - first < most ? p.sequences - first : most;
        const dim3 grid((unsigned)units, (unsigned)n, (unsigned)p.splits);
        auto with = [&](auto dim, auto scales) {
            constexpr int D = decltype(dim)::value, SCALES = decltype(scales)::value;
            if (wide) return attend_kernel<STORE, SCALES, D, true, 1><<<grid, kThreads, 0, s>>>(p, first);
            if constexpr (two_tiles(kHeadTile + 1, D, false)) {
                if (tiles == 2) return attend_kernel<STORE, SCALES, D, false, 2><<<grid, kThreads, 0, s>>>(p, first);
            }
            attend_kernel<STORE, SCALES, D, false, 1><<<grid, kThreads, 0, s>>>(p, first);
        };
        auto go = [&](auto dim) {
            if constexpr (STORE != kStoreBf16) {
                if (p.c.scales == kScaleRowF32) return with(dim, std::integral_constant<int, kScaleRowF32>{});
                if (p.c.scales == kScaleRowF16) return with(dim, std::integral_constant<int, kScaleRowF16>{});
            }
            with(dim, std::integral_constant<int, kScaleNone>{});
        };
        switch (p.c.head_dim) {
            case 64: go(std::integral_constant<int, 64>{}); break;
            case 96: go(std::integral_constant<int, 96>{}); break;
            case 128: go(std::integral_constant<int, 128>{}); break;
            case 192: go(std::integral_constant<int, 192>{}); break;
            default: go(std::integral_constant<int, 256>{}); break;
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace attend

hipError_t launch_attend_bf16(const AttendParams& p, hipStream_t s);
hipError_t launch_attend_e4m3(const AttendParams& p, hipStream_t s);
hipError_t launch_attend_e5m2(const AttendParams& p, hipStream_t s);
hipError_t launch_attend_e2m1(const AttendParams& p, hipStream_t s);

}  // namespace fp4
