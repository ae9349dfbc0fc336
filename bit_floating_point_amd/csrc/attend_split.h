// How the attention over a cache divides the positions of a sequence into parts: the host's
// choice of how many parts a launch has room for, and the device's choice of a part's
// positions.  Plain integers, no GPU.
#pragma once
#include <stdint.h>

#include "cache_place.h"

namespace fp4 {

constexpr int kTilePositions = 32;  // positions that a wavefront takes at a time
constexpr int kAttendWaves = 4;     // wavefronts of a workgroup, on tiles in turn
constexpr int kPartLeast = 512;     // positions of a part, at least (the last one aside)
constexpr int kMostSplits = 256;
constexpr int64_t kWantedWorkgroups = 1024;
constexpr int kHeadTile = 16;       // query heads of a workgroup

// positions that a sequence of up to `length` sees, from a multiple of a tile on
inline int64_t most_seen(int64_t length, int64_t window) {
    return window > 0 && window < length - kTilePositions ? window + kTilePositions - 1 : length;
}

// Parts per sequence: as many as bring the launch to kWantedWorkgroups, none of them shorter than
// kPartLeast.  Grows with max_length.
inline int32_t split_count(int64_t sequences, int32_t heads, int32_t kv_heads, int64_t max_length, int64_t window) {
    const int64_t tiles = (heads / kv_heads + kHeadTile - 1) / kHeadTile;
    const int64_t units = sequences * kv_heads * tiles;
    const int64_t parts = (most_seen(max_length, window) + kPartLeast - 1) / kPartLeast;
    int64_t s = (kWantedWorkgroups + units - 1) / units;
    if (s > parts) s = parts;
    if (s > kMostSplits) s = kMostSplits;
    return (int32_t)(s < 1 ? 1 : s);
}

// The positions [begin, end) that a sequence of n positions sees are divided from
// `first` = begin rounded down to a tile, `chunk` at a time; `used` parts have any.
struct SplitRange {
    int32_t begin, first, chunk, used;
};
FP4_HD inline SplitRange split_range(int32_t n, int32_t window, int32_t splits) {
    SplitRange r;
    r.begin = window > 0 && window < n ? n - window : 0;
    r.first = r.begin / kTilePositions * kTilePositions;
    const int32_t count = n - r.first;
    const int32_t step = kTilePositions * kAttendWaves;  // every wavefront gets as many tiles
    int32_t chunk = (count + splits - 1) / splits;
    chunk = chunk < kPartLeast ? kPartLeast : (int32_t)(((int64_t)chunk + step - 1) / step * step);
    r.chunk = chunk;
    r.used = count > 0 ? (count - 1) / chunk + 1 : 0;
    return r;
}

}  // namespace fp4
