// How the attention over a cache divides the positions of a sequence into parts: the host's
// choice of how many parts a launch has room for, and the device's choice of a part's
// positions.  Plain integers, no GPU.
#pragma once
#include <stdint.h>

#include "cache_place.h"

namespace fp4 {

constexpr int kTilePositions = 32;  // positions that a wavefront takes at a time
constexpr int kAttendWaves = 4;     // wavefronts of a workgroup, on tiles in turn
// Positions of a part, at least (the last one aside): 2^9, or 2^8 where all sequences and heads together are fewer workgroups than
// compute units, as far as that fills these once.  Shorter parts mean more to join, longer ones idle compute units (parts of
// 512 / of 256, us of the call, 8 kv heads with 8 heads each, E4M3: 1 sequence of 8192 11.1 / 9.6, of 2048 10.8 / 9.1, 4 of 1024 10.5 / 9.6,
// 1 of 2000 bf16 15.6 / 11.7; past the fill 1 of 16384 11.7 / 13.3, of 32768 18.7 / 21.8, 25 of 3000 38.0 / 39.6; with more
// units 64 of up to 700 13.7 / 18.3).  Below 1024 positions one part, which has no join, is still a little quicker than two:
// 8 of 1000 10.4 / 10.9, 2 of 800 9.1 / 10.0.
constexpr int kPartLeastLog = 9, kPartLeastFewLog = 8;
constexpr int64_t kFewUnits = 256;
constexpr int kMostSplits = 256;  // threads of a join's workgroup
// Four workgroups a compute unit.  1024 / 2048 / 4096, us: 16x4096 of 40 kv heads E4M3 113 / 131 / 150; 48x8192 of 8, 153 / 167 /
// 186, E2M1 84 / 95 / 104; 1x131072 bf16 86 / 90 / 91; lengths up to 8192, 96 sequences: E2M1 92 / 98 / 102, E4M3 200 / 190 /
// 194, bf16 341 / 330 / 337: even batches lose more by two than ragged ones gain.  (Tiles of query heads are counted one by one:
// a launch whose workgroups take two has half as many.)
constexpr int64_t kWantedWorkgroups = 1024;
constexpr int kHeadTile = 16;       // query heads of a tile: a workgroup takes one or two

// Positions that a sequence of up to `length` sees, from a multiple of a tile on: no more than the window and what lies
// before it in its first tile.
inline int64_t most_seen(int64_t length, int64_t window) {
    constexpr int64_t before = kTilePositions - 1;
    return window > 0 && window < length - before ? window + before : length;
}

// sequences, kv heads and tiles of their query heads
inline int64_t attend_units(int64_t sequences, int32_t heads, int32_t kv_heads) {
    return sequences * kv_heads * ((heads / kv_heads + kHeadTile - 1) / kHeadTile);
}

// How many parts a sequence gets: a power of two, as every workgroup divides by it.  One rule for the host, which makes room by the
// longest sequence that a call can have, and for the device, which goes by each sequence's own length: the room is what the
// longest one uses, and a sequence's parts are the same in every call that has as many units.
struct PartRule {
    int32_t few_log;  // up to 2^few_log parts may be as short as 2^kPartLeastFewLog
    // log2 of the parts of a sequence that sees `count` positions.  Up to 2^kPartLeastLog positions are one part always: they
    // need no join (1 sequence of 512, 32 kv heads: 7.0 us, in two parts 10.1).
    FP4_HD int32_t parts_log(int32_t count) const {
        if (count <= 1 << kPartLeastLog) return 0;
        const int32_t size = 31 - __builtin_clz((unsigned)count);
        const int32_t fit = size - kPartLeastFewLog, few = fit < few_log ? fit : few_log, more = size - kPartLeastLog;
        return few > more ? few : more;
    }
};
// the rule of a launch: short parts up to the first power of two that fills the compute units
inline PartRule part_least_log(int64_t units) {
    PartRule r{0};
    while (units << r.few_log < kFewUnits) r.few_log++;
    return r;
}

// Parts that a launch makes room for per sequence, a power of two: those of the longest sequence, as far as they bring it to
// kWantedWorkgroups.  Grows with max_length (at most 2^30).
inline int32_t split_count(int64_t sequences, int32_t heads, int32_t kv_heads, int64_t max_length, int64_t window) {
    const int64_t units = attend_units(sequences, heads, kv_heads);
    const int64_t parts = (int64_t)1 << part_least_log(units).parts_log((int32_t)most_seen(max_length, window));
    const int64_t wanted = (kWantedWorkgroups + units - 1) / units;
    int32_t s = 1;
    while (s < wanted && s < parts && s < kMostSplits) s *= 2;
    return s;
}

// The positions [begin, n) that a sequence of n positions sees are divided from `first` = begin
// rounded down to a tile, `chunk` at a time; `count` of them from there.
struct SplitRange {
    int32_t begin, first, count, chunk;
    FP4_HD int32_t used() const { return count > 0 ? (count - 1) / chunk + 1 : 0; }
    FP4_HD bool has(int32_t split) const { return (int64_t)split * chunk < count; }
};
// the sequence's parts by the rule, 2^split_log at most
FP4_HD inline SplitRange split_range(int32_t n, int32_t window, int32_t split_log, PartRule rule) {
    SplitRange r;
    r.begin = window > 0 && window < n ? n - window : 0;
    r.first = r.begin / kTilePositions * kTilePositions;
    r.count = n - r.first;
    const int32_t fit = rule.parts_log(r.count), log = fit < split_log ? fit : split_log;
    constexpr int32_t step = kTilePositions * kAttendWaves;  // every wavefront gets as many tiles
    const int32_t chunk = (int32_t)(((int64_t)r.count + (1 << log) - 1) >> log);
    r.chunk = chunk < step ? step : (chunk + step - 1) / step * step;
    return r;
}

}  // namespace fp4
