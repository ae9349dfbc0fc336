"""Where positions lie (csrc/cache_place.h) and how a sequence is divided (csrc/attend_split.h),
on the CPU under AddressSanitizer and UndefinedBehaviorSanitizer: tables of any content, positions
and sequence numbers at the ends of their types never read outside the table, and every division
covers what a sequence sees exactly once, within the parts that the host made room for."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_floating_point_amd", "csrc")

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "attend_split.h"
using namespace fp4;
static void need(bool ok, const char* what, long long a, long long b, long long c) {
    if (!ok) { std::printf("%s: %lld %lld %lld\n", what, a, b, c); std::abort(); }
}
static void places() {
    const int64_t sequences = 3, ld = 5;
    const int32_t pages = 7, page_log = 4, most[] = {0, 1, 4};
    for (int32_t max_pages : most) {
        std::vector<int32_t> table((sequences - 1) * ld + max_pages);  // ends with its last row
        const int32_t odd[] = {0, 6, 7, -1, INT32_MIN, INT32_MAX, 3};
        for (size_t i = 0; i < table.size(); i++) table[i] = odd[i % 7];
        const int32_t capacity = max_pages << page_log;
        const int64_t of[] = {0, 1, 2, 3, -1, INT32_MIN, INT32_MAX, INT64_MAX, INT64_MIN};
        for (int64_t s : of)
            for (int64_t t = -70; t < 70; t++) {
                const int64_t ends[] = {t, INT32_MIN - t, INT32_MAX + (t < 0 ? t : -t)};
                for (int64_t p64 : ends) {
                    if (p64 < INT32_MIN || p64 > INT32_MAX) continue;
                    const int32_t p = (int32_t)p64;
                    const RowPlace r = find_row(table.data(), sequences, ld, capacity, page_log, pages, s, p);
                    const bool there = s >= 0 && s < sequences && p >= 0 && p < capacity;
                    const int32_t page = there ? table[s * ld + p / 16] : -1;
                    const bool good = there && page >= 0 && page < pages;
                    need(r.page == (good ? page : -1) && (!good || r.slot == p % 16), "place", s, p, r.page);
                }
            }
    }
}
static void check(int64_t sequences, int32_t heads, int32_t kv_heads, int32_t most, int32_t window, int32_t n, bool each) {
    const int32_t splits = split_count(sequences, heads, kv_heads, most, window);
    need(splits >= 1 && splits <= kMostSplits, "splits", sequences, most, splits);
    need((splits & (splits - 1)) == 0, "power of two", sequences, most, splits);
    need(splits == 1 || most_seen(most, window) > 512, "short ones in one part", most, window, splits);
    const SplitRange r = split_range(n, window, __builtin_ctz(splits), part_least_log(attend_units(sequences, heads, kv_heads)));
    const int32_t parts = r.used();
    const int32_t begin = window > 0 && window < n ? n - window : 0;
    need(r.begin == begin && r.first <= begin && begin - r.first < kTilePositions && r.first % kTilePositions == 0, "begin", n, window, r.first);
    need(r.chunk > 0 && r.chunk % kTilePositions == 0, "chunk", n, splits, r.chunk);
    need(parts <= splits && (parts > 0) == (n > 0), "used", n, splits, parts);
    for (int32_t i = 0; i < splits; i++) need(r.has(i) == (i < parts), "has", n, i, parts);
    need(r.count == n - r.first && (parts > 1) == (r.count > r.chunk), "count", n, r.count, r.chunk);
    int64_t at = r.first;
    for (int32_t i = 0; i < parts; i++) {
        const int64_t b = r.first + (int64_t)i * r.chunk;
        const int32_t e = n - (int32_t)b < r.chunk ? n : (int32_t)b + r.chunk;  // the kernel's expression
        need(b == at && e > b && e <= n, "part", n, i, e);
        at = e;
        if (!each) continue;
        // the tiles of the wavefronts, by the kernel's counts
        const int all = (e - (int)b + kTilePositions - 1) / kTilePositions;
        int total = 0;
        for (int w = 0; w < kAttendWaves; w++) total += (all - w + kAttendWaves - 1) / kAttendWaves;
        need(total == all, "tiles", n, all, total);
    }
    need(n == 0 || at == n, "covered", n, splits, at);
}
int main() {
    places();
    for (int32_t n = 0; n < 3000; n++)
        for (int32_t window : {0, 1, 31, 33, 500, 1000, 5000}) {
            check(1, 8, 8, 3000, window, n, true);
            check(40, 5, 5, 3000, window, n, true);
        }
    const int32_t long_ones[] = {1 << 30, (1 << 30) - 1, (1 << 30) - 31, 1 << 29, 131072, 131073, 99999};
    for (int32_t most : long_ones)
        for (int32_t n : long_ones)
            for (int32_t window : {0, 1, 4097, 1 << 29, (1 << 30) - 1})
                for (int64_t sequences : {1ll, 3ll, 100ll, 0x7fffffffll})
                    if (n <= most) {
                        check(sequences, 40, 8, most, window, n, false);
                        check(sequences, 65536, 1, most, window, n, false);
                        check(sequences, 65535, 65535, most, window, n, false);
                    }
    std::puts("ok");
    return 0;
}
"""


def test_places_and_parts(tmp_path):
    (tmp_path / "p.cpp").write_text(SOURCE)
    exe = str(tmp_path / "p")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                           str(tmp_path / "p.cpp"), "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr[-2000:]
