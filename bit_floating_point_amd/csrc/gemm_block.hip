// Products of 8-bit operands whose scales change along K, and the experts' products:
//   Y[m, n] = T,  T = fma(P_b[m, n], fl32(sa[m, b] * sw[n / 128, b]), T) over the blocks b
// of 128 columns of K, P_b = sum over the block of the code products on the f8f6f4 matrix
// cores.  The scales differ from block to block, so a block's sum cannot stay in the
// accumulator of the next: every block ends in one fused multiply-add per output value, and
// T has to be in vector registers (the accumulation registers take no such instruction).
//
// Below binary32: within a block the matrix instruction drops product bits under 2^-13 of the
// largest product of 8, which is what its rate costs.  Binary32 results lie 1.5e-5 from the exact
// ones in norm for operands of even magnitudes, 4.6e-5 where 1 % of the channels are 50 times
// larger; of bf16 results, 3 % are the other neighbour of the exact value.
//
// The weight tile is the instruction's first operand, so a lane of a result holds columns n
// of one row m: both scales are one value per lane and block, and four consecutive columns
// leave in one store.
//
// Tile kernel (block_gemm_tile_kernel).  256 x 256 outputs on 8 wavefronts of 128 x 64: T takes
// 128 of a lane's 256 registers, the most that leaves two wavefronts per SIMD.  Operands go
// HBM -> LDS without registers, whole 128-byte lines (8 rows x 128 bytes an instruction), two
// stages of 128 codes; a stage's weights are replaced once every wavefront has them in
// registers, its activations at the step's end.  Scales come in chunks of 8 blocks: fetched one
// block at a time, each instruction touched 64 lines and they were a third of all L1 requests.
// 4096 x 15360 x 5120: 321 us (2.0 PFLOP/s; 8192^3 at 2.2; 357 with f32 results), where the library's product with one
// scale per tensor reaches 2.9 PFLOP/s at 8192^3; about 8 us of the 82 of a tile are its first
// loads and its output.  Bound by LDS: a step (2048 cycles of matrix
// instructions per SIMD) reads 192 KB of fragments and writes 64 KB, and each 1 KB read costs
// the SIMD's matrix cores about 18 cycles; the folds add about 500.  Measured at 8192^3 with parts
// left out: 505 us whole, 430 without loads, 370 without loads and folds.
// Smaller tiles and two wavefront groups per tile fill the chip on smaller grids (see
// gemm_block_choice.h); there a compute unit's load rate (57-70 GB/s) and the latency of a step bound.
//
// Streaming kernel (block_gemm_stream_kernel), few rows: bound by reading W.  1 x 11008 x 4096
// 11.1 us (4.1 TB/s with the launch), 1 x 15360 x 5120 14.2 us (5.5 TB/s), the 64 experts of 8
// tokens (881 MB) 122-138 us (6.4-7.2 TB/s).
//
// Experts: the list of slots (sorted by expert) is cut into m-tiles expert by expert, a
// workgroup finds its own from the offsets, and rows are gathered by the loads themselves.
// 4096 tokens x 8 of 64 experts, 4096 x 5120: 838 us (1.6 PFLOP/s): as above, with part of each
// expert's last tile unused (one that is half empty computes half: 898 -> 875 us) and the weights'
// 1.3 GB read beside.
#include <type_traits>

#include "fp4_device.h"
#include "gemm_block_choice.h"
#include "layer_internal.h"

namespace fp4 {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int FW, int FA>
__device__ __forceinline__ f32x16 mfma64(i32x8 w, i32x8 a, f32x16 c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, FW, FA, 0, 127, 0, 127);
}

template <int FW, int FA>
__device__ __forceinline__ f32x4 mfma128(i32x8 w, i32x8 a, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, FW, FA, 0, 127, 0, 127);
}

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// One store of v at an address that is aligned to ALIGN bytes only: the rows of y start where
// ldy puts them, and global stores take any alignment.
template <int ALIGN, typename T>
__device__ __forceinline__ void store_any(void* at, T v) {
    struct __attribute__((packed, aligned(ALIGN))) Loose { T v; };
    reinterpret_cast<Loose*>(at)->v = v;
}

__device__ __forceinline__ void store_y(const BlockGemmParams& p, int64_t row, int64_t col, float v) {
    if (p.y_bf16) reinterpret_cast<__bf16*>(p.y)[row * p.ldy + col] = (__bf16)v;
    else reinterpret_cast<float*>(p.y)[row * p.ldy + col] = v;
}

// four consecutive columns of a row, of which those below N are written
__device__ __forceinline__ void store_y4(const BlockGemmParams& p, int64_t row, int64_t col, float a, float b, float c, float d) {
    if (col + 4 <= p.N) {
        const int64_t at = row * p.ldy + col;
        if (p.y_bf16) {
            const bf16x4 v = {(__bf16)a, (__bf16)b, (__bf16)c, (__bf16)d};
            store_any<2>(reinterpret_cast<__bf16*>(p.y) + at, __builtin_bit_cast(uint2, v));
        } else {
            store_any<4>(reinterpret_cast<float*>(p.y) + at, make_float4(a, b, c, d));
        }
    } else {
        if (col < p.N) store_y(p, row, col, a);
        if (col + 1 < p.N) store_y(p, row, col + 1, b);
        if (col + 2 < p.N) store_y(p, row, col + 2, c);
    }
}

}  // namespace


// ---- tile kernel -----------------------------------------------------------------------
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Direct-to-LDS loads, 16 or 4 bytes per lane: lane l writes LDS bytes base + off + size l
// from the buffer at voff + soff (nothing, that is zeros, where voff is past the buffer).
__device__ __forceinline__ void lds_load16(i32x4v rsrc, uint32_t voff, uint32_t soff, uint32_t base, uint32_t off) {
    asm volatile("s_add_u32 m0, %2, %3\n\tbuffer_load_dwordx4 %0, %4, %1 offen lds"
                 :
                 : "v"(voff), "s"(soff), "s"(base), "s"(off), "s"(rsrc)
                 : "memory", "m0", "scc");
}
__device__ __forceinline__ void lds_load4(i32x4v rsrc, uint32_t voff, uint32_t soff, uint32_t base, uint32_t off) {
    asm volatile("s_add_u32 m0, %2, %3\n\tbuffer_load_dword %0, %4, %1 offen lds"
                 :
                 : "v"(voff), "s"(soff), "s"(base), "s"(off), "s"(rsrc)
                 : "memory", "m0", "scc");
}
#pragma clang diagnostic pop
// At most N of this wavefront's direct-to-LDS loads are in flight and its LDS reads have
// returned; then the workgroup barrier.
template <int N>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" : : "n"(N) : "memory");
}

// The m-tile and column block of a workgroup, in experts' mode its expert and slots.
struct Tile {
    int64_t e, lo, hi, m0;  // expert; its range of the list (dense: [0, M)); first row of the tile
    int n;                  // column block
    bool live;
};

// Workgroups go to the 8 XCDs in turn: XCD x takes the x-th eighth of the tiles, so that the
// tiles that share operands meet in one L2.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t ntiles) {
    const int64_t full = ntiles / 8 * 8;
    return b < full ? (b % 8) * (full / 8) + b / 8 : b;
}

// Offsets of any value are safe: ranges that overlap may hold more tiles than 32 bits count, so
// sums stop at 2^29.  Every tile that a workgroup may take lies below that, and so do the sums
// before it, which place it.
__device__ __forceinline__ int tile_sum(int a, int b) { return min(a + b, 1 << 29); }

template <int BM>
__device__ __forceinline__ Tile expert_tile(const BlockGemmParams& p, int grid_n) {
    const int lane = threadIdx.x & 63;
    auto range = [&](int e, int& lo, int& hi) {
        lo = hi = 0;
        if (e < p.experts) {
            lo = max(p.offsets[e], 0);
            hi = (int)min((int64_t)p.offsets[e + 1], p.M);
        }
        return hi > lo ? (hi - lo + BM - 1) / BM : 0;
    };
    int total = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
        int lo, hi, c = range(e0 + lane, lo, hi);
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) c = tile_sum(c, __shfl_xor(c, o, 64));
        total = tile_sum(total, c);
    }
    total = __builtin_amdgcn_readfirstlane(total);
    Tile t{};
    const int64_t ntiles = (int64_t)total * grid_n;
    if ((int64_t)blockIdx.x >= ntiles) return t;
    const int64_t at = xcd_order(blockIdx.x, ntiles);
    const int want = (int)(at / grid_n);
    int before = 0;
    for (int e0 = 0; e0 < p.experts; e0 += 64) {
        int lo, hi;
        const int c = range(e0 + lane, lo, hi);
        int s = c;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(s, o, 64);
            if (lane >= o) s = tile_sum(s, u);
        }
        const uint64_t hit = __ballot(before + s > want);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const int first = before + (l > 0 ? __shfl(s, l - 1, 64) : 0), mt = __shfl(c, l, 64);
            const int r = __builtin_amdgcn_readfirstlane((int)(at - (int64_t)first * grid_n));
            const int m = __builtin_amdgcn_readfirstlane(mt), from = __builtin_amdgcn_readfirstlane(__shfl(lo, l, 64));
            t.e = __builtin_amdgcn_readfirstlane(e0 + l);
            t.lo = from;
            t.hi = __builtin_amdgcn_readfirstlane(__shfl(hi, l, 64));
            t.m0 = from + (int64_t)(r % m) * BM;
            t.n = r / m;
            t.live = true;
            return t;
        }
        before = tile_sum(before, __shfl(s, 63, 64));
    }
    return t;
}

// S stages of 128 codes of K are in LDS or on their way there.
// A workgroup of WM x WN wavefronts computes BM x BN outputs, each wavefront MT x NT
// results of 32 x 32 (its m-tiles every WM-th of the tile's, so that a short tile's rows
// spread over the wavefronts).  KG such groups of wavefronts share a tile: group g takes the
// blocks g, KG + g, ... of K with stages of its own, and the sums are added in order at the
// end -- for grids that leave a compute unit one workgroup, whose steps would follow each
// other with nothing beside them.
template <int FW, int FA, int BM, int BN, int WM, int WN, int S, int KG, bool EXP>
__global__ void __launch_bounds__(64 * WM * WN * KG, 2) block_gemm_tile_kernel(BlockGemmParams p, int grid_m, int grid_n) {
    constexpr int NW = WM * WN, MT = BM / WM / 32, NT = BN / WN / 32;
    constexpr int SA = BM * 128, SB = BN * 128, STAGE = SA + SB;
    // scales: chunks of 8 blocks of K, BM rows (and the column blocks of W) of 8 values
    constexpr int CH = BM * 32 + 256 * (NW - BM / 64), NCH = 2;
    constexpr int LA = SA / 1024 / NW, LB = SB / 1024 / NW;
    static_assert(S == 2, "the counted waits and the scales' two chunks are for two stages");
    static_assert(BM / 64 < NW, "one wavefront per 64 scales of A, one for those of W");
    constexpr int REGION = S * STAGE + (NCH * CH + 1023) / 1024 * 1024;  // of one group
    __shared__ __attribute__((aligned(1024))) uint8_t smem_all[KG * REGION];
    __shared__ uint32_t scale_row[BM + 64];  // byte offset of the scales of each row, then of each column block

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) % NW);  // within its group
    const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane((threadIdx.x >> 6) / NW);
    uint8_t* const smem = smem_all + kg * REGION;
    uint8_t* const smem_s = smem + S * STAGE;
    const int wm = wave % WM, wn = wave / WM;
    const int r32 = lane & 31, hk = lane >> 5;

    Tile tile;
    if constexpr (EXP) {
        tile = expert_tile<BM>(p, grid_n);
        if (!tile.live) return;
    } else {
        // panels of four row blocks, column by column: the tiles that an XCD computes at
        // one time form a compact block
        const int64_t t = xcd_order(blockIdx.x, (int64_t)grid_m * grid_n);
        constexpr int P = 4;
        const int panel = (int)(t / ((int64_t)P * grid_n)), rows = min(P, grid_m - panel * P);
        const int r = (int)(t - (int64_t)panel * P * grid_n);
        tile.e = 0;
        tile.lo = 0;
        tile.hi = p.M;
        tile.m0 = (int64_t)(panel * P + r % rows) * BM;
        tile.n = r / rows;
    }
    const int64_t n0 = (int64_t)tile.n * BN;
    const int kb = (int)((p.K + 127) / 128), K = (int)p.K;
    const int steps = (kb + KG - 1) / KG;  // step b of group g is block b KG + g
    // output row and source row of the tile's row r, or -1
    auto rows_of = [&](int r, int64_t& src) -> int64_t {
        const int64_t m = tile.m0 + r;
        if (m >= tile.hi) return -1;
        if constexpr (!EXP) {
            src = r;  // from the tile's first row
            return m;
        } else {
            const int64_t s = p.slot_list[m];
            if (s < 0 || s >= p.M) return -1;
            src = s / p.slots_per_row;
            return s;
        }
    };

    // loads: LDS row r holds 8 pieces of 16 bytes, piece s at position s ^ (r / 2 % 8), so
    // that the 16 rows a fragment read serves at once lie in different banks
    const int64_t a_rows = EXP ? (p.M + p.slots_per_row - 1) / p.slots_per_row : min((int64_t)BM, p.M - tile.m0);
    const i32x4v rsA = buf_words(EXP ? p.a : p.a + tile.m0 * p.lda, a_rows * p.lda);
    const i32x4v rsB = buf_words(p.w + tile.e * p.stride_w + n0 * p.ldw, min((int64_t)BN, p.N - n0) * p.ldw);
    // scales: wavefront w < BM / 64 those of 64 rows of A, the next one those of W's blocks
    const int64_t nb0 = n0 / 128, nbs = min((int64_t)((BN + 127) / 128), (p.N + 127) / 128 - nb0);
    const bool of_a = wave < BM / 64;
    const i32x4v rsS = of_a ? buf_words(EXP ? p.a_scales : p.a_scales + tile.m0 * p.lda_s, a_rows * p.lda_s * 4)
                            : buf_words(p.w_scales + tile.e * p.stride_ws + nb0 * p.ldw_s, nbs * p.ldw_s * 4);
    const int seg = (lane & 7) ^ ((4 * (wave & 1) + (lane >> 4)) & 7);
    // dense operands: one offset per lane, the later pieces by the scalar offset.  Rows past the
    // operand read zeros: without a stride or swizzle a buffer's range check covers the sum of
    // both offsets (out of range where the lane's offset >= num_records - the scalar one: the
    // CDNA3 instruction set manual, range checking of buffer accesses), also where the scalar
    // offset alone is past the end.  Measured so on gfx950 for these loads into LDS and for
    // register loads of 4 and 16 bytes, on a descriptor shorter than its allocation.
    uint32_t offA[EXP ? LA : 1], offB;
    const int r8 = wave * 8 + (lane >> 3);
    if constexpr (EXP) {
#pragma unroll
        for (int i = 0; i < LA; i++) {
            int64_t src = 0;
            const int64_t out = rows_of(NW * 8 * i + r8, src);
            offA[i] = out < 0 ? kOOB : (uint32_t)(src * p.lda + seg * 16);
        }
    } else {
        offA[0] = (uint32_t)(r8 * (int)p.lda + seg * 16);
    }
    offB = (uint32_t)(r8 * (int)p.ldw + seg * 16);
    const uint32_t stepA = (uint32_t)(NW * 8 * (int)p.lda), stepB = (uint32_t)(NW * 8 * (int)p.ldw);
    for (int r = threadIdx.x; r < BM + 64; r += 64 * NW * KG) {
        int64_t src = r - BM;
        if (r < BM) scale_row[r] = rows_of(r, src) < 0 ? kOOB : (uint32_t)(src * p.lda_s * 4);
        else scale_row[r] = src < nbs ? (uint32_t)(src * p.ldw_s * 4) : kOOB;
    }
    const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
    const uint32_t lds_wave = __builtin_amdgcn_readfirstlane(lds + wave * 1024);
    const uint32_t lds_scale = __builtin_amdgcn_readfirstlane(lds + S * STAGE + wave * 256);
    // Pieces past K read zeros, and so do whole stages past it (the loop has no branch).
    auto load_a = [&](int b, uint32_t stage) {
        const uint32_t k = (uint32_t)((b * KG + kg) * 128), dead = (int)k + seg * 16 < K ? 0u : kOOB;
#pragma unroll
        for (int i = 0; i < LA; i++) {
            if constexpr (EXP) lds_load16(rsA, offA[i] |= dead, k, lds_wave, stage + NW * i * 1024);
            else lds_load16(rsA, offA[0] |= dead, k + i * stepA, lds_wave, stage + NW * i * 1024);
        }
    };
    auto load_w = [&](int b, uint32_t stage) {
        const uint32_t k = (uint32_t)((b * KG + kg) * 128), dead = (int)k + seg * 16 < K ? 0u : kOOB;
#pragma unroll
        for (int i = 0; i < LB; i++) lds_load16(rsB, offB |= dead, k + i * stepB, lds_wave, stage + SA + NW * i * 1024);
    };
    // Part c (of 8) of the scales' chunk q (of steps 8 q .. 8 q + 7): 8 values of BM / 8 rows,
    // and with every part those of W.  A load instruction then touches 8 lines, not 64.
    // Step k's of row r sits at position k ^ (r / 8 % 8): the reads of 32 rows fall into
    // different banks.
    auto load_scales = [&](int q, int c) {
        const int group = BM / 64 * c + wave;  // of 8 rows
        const uint32_t row = scale_row[(of_a ? 8 * group : BM + 8 * (wave - BM / 64)) + (lane >> 3)];
        const int k = (q * 8 + ((lane & 7) ^ (of_a ? group & 7 : 0))) * KG + kg;
        lds_load4(rsS, (row + (uint32_t)k * 4) | (k < kb ? 0u : kOOB), 0, lds_scale,
                  (uint32_t)(q % NCH) * CH + (of_a ? BM * 4 * c : BM * 28));
    };

    // fragment h (64 codes) of LDS row `row`: pieces 4 h + 2 hk and the next
    const int x = (r32 >> 1) & 7;
    auto frag = [&](const uint8_t* rows, int row, int h) -> i32x8 {
        const uint8_t* q = rows + (row + r32) * 128;
        const uint4 u = *reinterpret_cast<const uint4*>(q + (((4 * h + 2 * hk) ^ x) << 4));
        const uint4 v = *reinterpret_cast<const uint4*>(q + (((4 * h + 2 * hk + 1) ^ x) << 4));
        return i32x8{(int)u.x, (int)u.y, (int)u.z, (int)u.w, (int)v.x, (int)v.y, (int)v.z, (int)v.w};
    };

    f32x16 t[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++) t[i][j] = f32x16{};

    // A step's loads: the stage S steps ahead, and a part of the scales' chunk that has landed
    // before the chunk's first use.
    constexpr int GROUP = LA + LB + 1;
    auto load_rest = [&](int b, uint32_t stage) {
        load_w(b + S, stage);
        load_scales(((b + S - 1) >> 3) + 1, (b + S - 1) & 7);
    };
    load_w(0, 0);
    load_a(0, 0);
    __syncthreads();  // the table of scale rows
#pragma unroll
    for (int c = 0; c < 8; c++) load_scales(0, c);
    // (every stage but the first brings GROUP loads, as in the loop: the waits count them)
#pragma unroll
    for (int q = 1; q < S; q++) {
        load_w(q, q * STAGE);
        load_scales(1, q - 1);
        load_a(q, q * STAGE);
    }
    step_barrier<(S - 1) * GROUP>();
    // LIVE m-tiles of each wavefront have rows
    auto run = [&](auto live) {
        constexpr int LIVE = decltype(live)::value;
        uint32_t cur = 0;
        for (int b = 0; b < steps; b++) {
            const uint8_t* sa = smem + cur;
            const uint8_t* sb = sa + SA;
            const float* sc = reinterpret_cast<const float*>(smem_s + ((b >> 3) % NCH) * CH);
            const int c8 = b & 7;
            const float sw = sc[BM * 8 + (wn * NT * 32) / 128 * 8 + c8];
            i32x8 w[NT][2];
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int h = 0; h < 2; h++) w[j][h] = frag(sb, (wn * NT + j) * 32, h);
            i32x8 a[2];
#pragma unroll
            for (int h = 0; h < 2; h++) a[h] = frag(sa, wm * 32, h);
            f32x16 c[NT];
            float s[LIVE];
#pragma unroll
            for (int i = 0; i < LIVE; i++) s[i] = sc[((i * WM + wm) * 32 + r32) * 8 + (c8 ^ (((i * WM + wm) * 4 + (r32 >> 3)) & 7))] * sw;
            // m-tile i: the first halves of its NT block sums, then the second; a sum is folded
            // into t while the matrix cores work on the next one
            auto fold = [&](int i, int j) {
#pragma unroll
                for (int v = 0; v < 16; v++) t[i][j][v] = __builtin_fmaf(c[j][v], s[i], t[i][j][v]);
            };
#pragma unroll
            for (int i = 0; i < LIVE; i++) {
                if (i == 1 && LIVE > 2) {
                    // every wavefront has read this stage's weights: those S steps on replace them
                    step_barrier<S * GROUP>();
                    load_rest(b, cur);
                    __builtin_amdgcn_sched_barrier(0);
                }
                if (i + 1 == LIVE) {
                    // every fragment of this stage is read (by all wavefronts, past the barrier)
                    // and the next stage's loads have landed
                    if constexpr (LIVE > 2) {
                        step_barrier<LB + 1>();
                    } else {
                        step_barrier<0>();
                        load_rest(b, cur);
                    }
                    load_a(b + S, cur);
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    if (i > 0 && j + 1 == NT) fold(i - 1, NT - 1);
                    c[j] = mfma64<FW, FA>(w[j][0], a[0], f32x16{});
                }
                if (i + 1 < LIVE) a[0] = frag(sa, ((i + 1) * WM + wm) * 32, 0);
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    c[j] = mfma64<FW, FA>(w[j][1], a[1], c[j]);
                    if (j > 0) fold(i, j - 1);
                }
                if (i + 1 < LIVE) a[1] = frag(sa, ((i + 1) * WM + wm) * 32, 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            fold(LIVE - 1, NT - 1);
            cur = cur + STAGE == S * STAGE ? 0 : cur + STAGE;
        }
    };
    // an expert's last tile is half empty as often as not
    if (EXP && MT > 2 && tile.hi - tile.m0 <= BM / 2) run(std::integral_constant<int, MT / 2>{});
    else run(std::integral_constant<int, MT>{});
    step_barrier<0>();  // no load into LDS outlives the workgroup

    if constexpr (KG > 1) {
        float4* part = reinterpret_cast<float4*>(smem_all);
        auto at = [&](int g, int i, int j, int q) { return ((((g - 1) * NW + wave) * MT + i) * NT + j) * 4 + q; };
        if (kg > 0) {
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        part[at(kg, i, j, q) * 64 + lane] =
                            make_float4(t[i][j][4 * q], t[i][j][4 * q + 1], t[i][j][4 * q + 2], t[i][j][4 * q + 3]);
        }
        __syncthreads();
        if (kg > 0) return;
#pragma unroll
        for (int g = 1; g < KG; g++)
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < NT; j++)
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const float4 v = part[at(g, i, j, q) * 64 + lane];
                        t[i][j][4 * q] += v.x;
                        t[i][j][4 * q + 1] += v.y;
                        t[i][j][4 * q + 2] += v.z;
                        t[i][j][4 * q + 3] += v.w;
                    }
    }

    if (p.y_bf16) {
        // The stages are free now: each wavefront turns its results to rows in LDS of its own
        // and writes 16 bytes per lane, whole lines of several rows at a time.  (Stores of
        // four columns straight from the results touch 32 rows an instruction: 4 us more per
        // 256 x 256 tile.)
        constexpr int COLS = NT * 32, PITCH = COLS * 2 + 16, LANES = COLS / 8, ROWS = 64 / LANES;
        // behind the other groups' sums, which slower wavefronts may still be reading
        constexpr int PARTS = (KG - 1) * NW * MT * NT * 4 * 64 * 16;
        static_assert(PARTS + NW * MT * 32 * PITCH <= KG * REGION, "the wavefronts' rows fit the stages");
        uint8_t* mine = smem_all + PARTS + wave * (MT * 32 * PITCH);
#pragma unroll
        for (int i = 0; i < MT; i++)
#pragma unroll
            for (int j = 0; j < NT; j++)
#pragma unroll
                for (int q = 0; q < 4; q++)
                    *reinterpret_cast<bf16x4*>(mine + (i * 32 + r32) * PITCH + (j * 32 + 8 * q + 4 * hk) * 2) =
                        bf16x4{(__bf16)t[i][j][4 * q], (__bf16)t[i][j][4 * q + 1], (__bf16)t[i][j][4 * q + 2], (__bf16)t[i][j][4 * q + 3]};
        const int64_t col = n0 + wn * COLS + (lane % LANES) * 8;
#pragma unroll 4
        for (int r0 = 0; r0 < MT * 32; r0 += ROWS) {
            const int r = r0 + lane / LANES;
            int64_t src = 0;
            const int64_t out = rows_of(((r >> 5) * WM + wm) * 32 + (r & 31), src);
            const uint4 v = *reinterpret_cast<const uint4*>(mine + r * PITCH + (lane % LANES) * 16);
            if (out < 0) continue;
            __bf16* y = reinterpret_cast<__bf16*>(p.y) + out * p.ldy + col;
            if (col + 8 <= p.N) {
                store_any<2>(y, v);
            } else {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (col + e < p.N) reinterpret_cast<uint16_t*>(y)[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < MT; i++) {
        int64_t src = 0;
        const int64_t out = rows_of((i * WM + wm) * 32 + r32, src);
        if (out < 0) continue;
#pragma unroll
        for (int j = 0; j < NT; j++)
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int64_t col = n0 + (wn * NT + j) * 32 + 8 * g + 4 * hk;
                store_y4(p, out, col, t[i][j][4 * g], t[i][j][4 * g + 1], t[i][j][4 * g + 2], t[i][j][4 * g + 3]);
            }
    }
}

// ---- few rows ----------------------------------------------------------------------------
// Reading the weights is what the product costs.  A workgroup computes 16 MT rows of A by
// 16 NT rows of W; its KS wavefronts take the blocks of K between them, each streaming its
// operands straight into fragments, D blocks ahead, and the KS partial sums are added in
// order through LDS.  The 16 x 16 x 128 instruction takes a whole block, so its result is
// the block's sum.
template <int FW, int FA, int MT, int NT, int KS, int D, bool EXP>
__global__ void __launch_bounds__(64 * KS, 2) block_gemm_stream_kernel(BlockGemmParams p, int grid_m, int grid_n) {
    constexpr int BM = 16 * MT, BN = 16 * NT;
    __shared__ f32x4 part[KS][MT * NT][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, g = lane >> 4;

    Tile tile;
    if constexpr (EXP) {
        tile = expert_tile<BM>(p, grid_n);
        if (!tile.live) return;
    } else {
        tile.e = 0;
        tile.lo = 0;
        tile.hi = p.M;
        tile.m0 = (int64_t)(blockIdx.x % grid_m) * BM;
        tile.n = blockIdx.x / grid_m;
    }
    const int64_t n0 = (int64_t)tile.n * BN;
    const int kb = (int)((p.K + 127) / 128), K = (int)p.K;
    const int64_t a_rows = EXP ? (p.M + p.slots_per_row - 1) / p.slots_per_row : min((int64_t)BM, p.M - tile.m0);
    const __amdgpu_buffer_rsrc_t rA = buf_make(EXP ? p.a : p.a + tile.m0 * p.lda, a_rows * p.lda);
    const __amdgpu_buffer_rsrc_t rS = buf_make(EXP ? p.a_scales : p.a_scales + tile.m0 * p.lda_s, a_rows * p.lda_s * 4);
    const __amdgpu_buffer_rsrc_t rW = buf_make(p.w + tile.e * p.stride_w + n0 * p.ldw, min((int64_t)BN, p.N - n0) * p.ldw);
    const __amdgpu_buffer_rsrc_t rV = buf_make(p.w_scales + tile.e * p.stride_ws + n0 / 128 * p.ldw_s, (int64_t)kb * 4);
    int64_t out[MT];
    uint32_t offA[MT], offS[MT];
#pragma unroll
    for (int i = 0; i < MT; i++) {
        const int64_t m = tile.m0 + 16 * i + r16;
        int64_t src = 16 * i + r16;
        out[i] = m < tile.hi ? m : -1;
        if constexpr (EXP) {
            if (out[i] >= 0) out[i] = p.slot_list[m];
            if (out[i] >= p.M) out[i] = -1;
            src = out[i] / p.slots_per_row;
        }
        offA[i] = out[i] < 0 ? kOOB : (uint32_t)(src * p.lda + 16 * g);
        offS[i] = out[i] < 0 ? kOOB : (uint32_t)(src * p.lda_s * 4);
    }
    const uint32_t offW = (uint32_t)(r16 * (int)p.ldw + 16 * g);

    struct Stage {
        i32x8 w[NT], a[MT];
        float sa[MT], sw;
    } st[D];
    // A lane's 32 codes of a block: pieces g and 4 + g of 16 (any assignment of codes to lanes
    // that both operands share gives the block's sum; with this one the four lanes of a row
    // read 64 contiguous bytes).
    auto load32 = [&](__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t soff, uint32_t d0, uint32_t d1) -> i32x8 {
        const auto u = __builtin_amdgcn_raw_buffer_load_b128(r, off | d0, soff, 0);
        const auto v = __builtin_amdgcn_raw_buffer_load_b128(r, (off + 64) | d1, soff, 0);
        return i32x8{(int)u[0], (int)u[1], (int)u[2], (int)u[3], (int)v[0], (int)v[1], (int)v[2], (int)v[3]};
    };
    const int per = (kb + KS - 1) / KS, first = wave * per, end = min(first + per, kb);
    // block b: zeros past K and past this wavefront's range
    auto load = [&](Stage& s, int b) {
        const uint32_t k = (uint32_t)b * 128;
        const uint32_t d = b < end ? 0u : kOOB;
        const uint32_t d0 = d | ((int)k + 16 * g < K ? 0u : kOOB), d1 = d | ((int)k + 16 * g + 64 < K ? 0u : kOOB);
#pragma unroll
        for (int j = 0; j < NT; j++) s.w[j] = load32(rW, offW, k + 16 * j * (uint32_t)p.ldw, d0, d1);
        s.sw = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rV, d, b * 4, 0));
#pragma unroll
        for (int i = 0; i < MT; i++) {
            s.a[i] = load32(rA, offA[i], k, d0, d1);
            s.sa[i] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rS, offS[i] | d, b * 4, 0));
        }
    };
    f32x4 t[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++) t[i][j] = f32x4{};
#pragma unroll
    for (int d = 0; d < D; d++) load(st[d], first + d);
    for (int b = first; b < end; b += D) {
#pragma unroll
        for (int d = 0; d < D; d++) {
#pragma unroll
            for (int i = 0; i < MT; i++) {
                const float s = st[d].sa[i] * st[d].sw;
#pragma unroll
                for (int j = 0; j < NT; j++) {
                    const f32x4 c = mfma128<FW, FA>(st[d].w[j], st[d].a[i], f32x4{});
#pragma unroll
                    for (int v = 0; v < 4; v++) t[i][j][v] = __builtin_fmaf(c[v], s, t[i][j][v]);
                }
            }
            load(st[d], b + d + D);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; i++)
#pragma unroll
        for (int j = 0; j < NT; j++) part[wave][i * NT + j][lane] = t[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; i++) {
#pragma unroll
        for (int j = 0; j < NT; j++) {
            if ((i * NT + j) % KS != wave) continue;
            f32x4 v = part[0][i * NT + j][lane];
#pragma unroll
            for (int q = 1; q < KS; q++) v += part[q][i * NT + j][lane];
            if (out[i] >= 0) store_y4(p, out[i], n0 + 16 * j + 4 * g, v[0], v[1], v[2], v[3]);
        }
    }
}

// launch(part, grid_m, grid_n) for the product, in as few parts as launches allow: ranges of
// column blocks that begin on a scale block of W, and for dense operands of row blocks.
// (Experts: tiles_m is the most that any layout takes, and stays below a launch's limit.)
template <int BM, int BN, typename Launch>
static hipError_t in_parts(const BlockGemmParams& p, int64_t tiles_m, int threads, Launch launch) {
    constexpr int64_t U = BN < kBlock ? kBlock / BN : 1;  // column blocks of a scale block
    const int64_t most = max_workgroups(threads), tiles_n = (p.N + BN - 1) / BN;
    const int64_t fit = most / (tiles_n < U ? tiles_n : U), gm = p.experts || tiles_m < fit ? tiles_m : fit;
    const int64_t gn = tiles_n <= most / gm ? tiles_n : most / gm / U * U;
    for (int64_t m = 0; m < tiles_m; m += gm) {
        for (int64_t n = 0; n < tiles_n; n += gn) {
            BlockGemmParams q = p;
            const int64_t row = m * BM, col = n * BN, tm = tiles_m - m < gm ? tiles_m - m : gm, tn = tiles_n - n < gn ? tiles_n - n : gn;
            if (!p.experts) q.M = p.M - row < tm * BM ? p.M - row : tm * BM;
            q.N = p.N - col < tn * BN ? p.N - col : tn * BN;
            q.a += row * p.lda;
            q.a_scales += row * p.lda_s;
            q.w += col * p.ldw;
            q.w_scales += col / kBlock * p.ldw_s;
            q.y = reinterpret_cast<uint8_t*>(p.y) + (row * p.ldy + col) * (p.y_bf16 ? 2 : 4);
            launch(q, tm, tn);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
    }
    return hipSuccess;
}

// m-tiles of BM rows: those of the experts' lists however the slots fall
static int64_t m_tiles(const BlockGemmParams& p, int64_t bm) {
    return p.experts ? p.M / bm + (p.experts < p.M ? p.experts : p.M) : (p.M + bm - 1) / bm;
}

template <int FW, int FA, int MT, int NT, int KS, int D>
static hipError_t launch_stream(const BlockGemmParams& p, hipStream_t s) {
    constexpr int threads = 64 * KS;
    return in_parts<16 * MT, 16 * NT>(p, m_tiles(p, 16 * MT), threads, [&](const BlockGemmParams& q, int64_t gm, int64_t gn) {
        if (q.experts) block_gemm_stream_kernel<FW, FA, MT, NT, KS, D, true><<<(unsigned)(gm * gn), threads, 0, s>>>(q, 0, (int)gn);
        else block_gemm_stream_kernel<FW, FA, MT, NT, KS, D, false><<<(unsigned)(gm * gn), threads, 0, s>>>(q, (int)gm, (int)gn);
    });
}

template <int FW, int FA, int BM, int BN, int WM, int WN, int S, int KG = 1>
static hipError_t launch_tiles(const BlockGemmParams& p, hipStream_t s) {
    constexpr int threads = 64 * WM * WN * KG;
    return in_parts<BM, BN>(p, m_tiles(p, BM), threads, [&](const BlockGemmParams& q, int64_t gm, int64_t gn) {
        if (q.experts) block_gemm_tile_kernel<FW, FA, BM, BN, WM, WN, S, KG, true><<<(unsigned)(gm * gn), threads, 0, s>>>(q, 0, (int)gn);
        else block_gemm_tile_kernel<FW, FA, BM, BN, WM, WN, S, KG, false><<<(unsigned)(gm * gn), threads, 0, s>>>(q, (int)gm, (int)gn);
    });
}

template <int FW, int FA>
static hipError_t launch_formats(const BlockGemmParams& p, hipStream_t s) {
    switch (block_kernel(p.experts, p.M, p.N)) {
        case BlockKernel::kStream16: return launch_stream<FW, FA, 1, 1, 4, 2>(p, s);
        case BlockKernel::kStream32: return launch_stream<FW, FA, 1, 2, 4, 2>(p, s);
        case BlockKernel::kStream64: return launch_stream<FW, FA, 1, 4, 4, 2>(p, s);
        case BlockKernel::kTile64K4: return launch_tiles<FW, FA, 64, 64, 1, 2, 2, 4>(p, s);
        case BlockKernel::kTile64K2: return launch_tiles<FW, FA, 64, 64, 1, 2, 2, 2>(p, s);
        case BlockKernel::kTile128K2: return launch_tiles<FW, FA, 128, 128, 2, 2, 2, 2>(p, s);
        case BlockKernel::kTile128: return launch_tiles<FW, FA, 128, 128, 2, 2, 2>(p, s);
        case BlockKernel::kTile256: break;
    }
    return launch_tiles<FW, FA, 256, 256, 2, 4, 2>(p, s);
}

hipError_t launch_gemm_block(const BlockGemmParams& p, hipStream_t s) {
    if (p.fw == 0) return p.fa == 0 ? launch_formats<0, 0>(p, s) : launch_formats<0, 1>(p, s);
    return p.fa == 0 ? launch_formats<1, 0>(p, s) : launch_formats<1, 1>(p, s);
}

}  // namespace fp4
