// Which kernel a block-scaled product runs (gemm_block.hip), by its sizes alone.
#pragma once
#include <cmath>
#include <cstdint>

namespace fp4 {

enum class BlockKernel {
    kStream16,   // streaming, 16, 32 or 64 columns a workgroup
    kStream32,
    kStream64,
    kTile64K4,   // tiles of 64 x 64, four or two groups of wavefronts taking K in turn
    kTile64K2,
    kTile128K2,  // tiles of 128 x 128, two groups or one
    kTile128,
    kTile256,    // tiles of 256 x 256
};

// Which kernel (us, measured one against the other).
// Up to 16 rows the streaming kernel, as wide in N as leaves 150 workgroups: A is read once per
// workgroup (16 / 32 / 64 columns: 5120 x 5120, one row 11.6 / 7.7 / 12.4; 11008 x 4096: 13.8 /
// 11.3 / 11.1; 4096 x 13824, four rows 12.6 / 18.4 / 30.3).  At 17 rows and more the tiles win
// (24 x 11008 x 4096: 13.5 against 15.9).
// Tiles: a step of 128 of K takes about 2.0 us with a 256 x 256 tile on every compute unit, 1.2
// with two 128 x 128 ones, 0.7 with one (two groups of wavefronts), 0.44 with two 64 x 64 ones
// (two groups each) and 0.22 with one (four groups: 64 x 4096 x 4096 10.5 against 11.4 with two,
// but 203 x 4100 x 2080, 260 tiles, 16.9 against 11.4); the least total wins (64 / 128 / 256:
// 203 x 4100 x 2080 11 / 16 / 33; 1024 x 4096 x 4096 33 / 25 / 52; 2048 x 4096 x 4096 66 / 41 / 59;
// 4096 x 15360 x 5120 604 / 390 / 356).
// Experts: lists of the mean length, each with half a tile to spare.  They are bound by reading
// the experts' weights until the lists are long: streaming up to four rows a list (64 experts of
// 4096 x 4096, streamed / tiles: one row 188 / 193, four 187 / 189, eight 191 / 189), then
// 128 x 128 tiles against 256 x 256 ones, the smaller tiles only where those leave compute units
// idle (8 rows: 187 against 211 with 64 x 64).  One long list among short ones does not turn the
// order round, though its weights are streamed once per 16 rows: 256 slots, 128 of them in one
// list 193 / 211, 192 of them 202 / 209.
inline BlockKernel block_kernel(int32_t experts, int64_t M, int64_t N) {
    const double lists = experts ? (double)(experts < M ? experts : M) : 1.0, rows = (double)M / lists;
    if (rows <= (experts ? 4 : 16)) {
        const double columns = lists * (double)N;
        return columns >= 64 * 150 ? BlockKernel::kStream64 : columns >= 32 * 150 ? BlockKernel::kStream32 : BlockKernel::kStream16;
    }
    auto tiles = [&](int b) {
        const double m = experts ? lists * std::fmax(1.0, rows / b + 0.5) : (double)((M + b - 1) / b);
        return m * (double)((N + b - 1) / b);
    };
    auto steps = [&](int b, double one, double two) { return tiles(b) <= 256 ? one : two * std::ceil(tiles(b) / 512); };
    const double t256 = 2.0 * std::ceil(tiles(256) / 256), t128 = steps(128, 0.7, 1.2), t64 = steps(64, 0.22, 0.44);
    const bool small = t64 < t128 && !(experts && tiles(128) > 256);
    if (t256 <= t128 && !(small && t64 < t256)) return BlockKernel::kTile256;
    if (small) return tiles(64) <= 256 ? BlockKernel::kTile64K4 : BlockKernel::kTile64K2;
    return tiles(128) <= 256 ? BlockKernel::kTile128K2 : BlockKernel::kTile128;
}

}  // namespace fp4
