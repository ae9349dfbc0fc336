"""How many parts the attention over a cache makes of a sequence (csrc/attend_split.h), on the CPU: by what that sequence sees
and by how many workgroups the launch has without parts, whatever longer sequences the call has room for; and
the host makes room for no part that no sequence can have."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_floating_point_amd", "csrc")

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "attend_split.h"
using namespace fp4;
struct Call { int64_t sequences; int32_t heads, kv_heads; };
static int64_t units_of(const Call& c) { return attend_units(c.sequences, c.heads, c.kv_heads); }
// The rule, by trial: the most parts, a power of two, that leave 512 positions to each, or 256 while
// the parts before the last doubling did not fill 256 compute units; one for 512 positions or fewer.
static int32_t parts_of(int64_t units, int64_t count) {
    int32_t best = 1;
    for (int32_t p = 2; p <= 256 && count > 512; p *= 2)
        if (count / p >= 512 || (count / p >= 256 && units * (p / 2) < 256)) best = p;
    return best;
}
static void need(bool ok, const char* what, const Call& c, long long most, long long n, long long window, long long got) {
    if (ok) return;
    std::printf("%s: %lld units, max_length %lld, length %lld, window %lld: %lld\n", what, (long long)units_of(c), most, n, window, got);
    std::exit(1);
}
int main() {
    const Call calls[] = {{1, 8, 8}, {1, 32, 32}, {5, 8, 8}, {25, 8, 8}, {33, 15, 5}, {31, 64, 8}, {32, 8, 8}, {64, 8, 8}, {300, 5, 5}, {1, 1, 1}, {1, 64, 1}};
    const int32_t lengths[] = {1, 31, 511, 512, 513, 700, 1000, 1023, 1024, 1025, 1400, 2000, 2048, 3000, 4096, 8191, 8192, 16384, 32768, 70000, 131072, 1 << 20};
    for (const Call& c : calls) {
        const int64_t units = units_of(c), wanted = (1024 + units - 1) / units;
        int32_t most_parts = 1;  // the power of two that the wanted workgroups need
        while (most_parts < wanted) most_parts *= 2;
        if (most_parts > 256) most_parts = 256;
        for (int32_t window : {0, 300, 481, 993, 1000, 3000, 20000})
            for (int32_t most : lengths) {
                const int32_t splits = split_count(c.sequences, c.heads, c.kv_heads, most, window);
                const int32_t rule = parts_of(units, most_seen(most, window));
                need(splits == (rule < most_parts ? rule : most_parts), "room", c, most, most, window, splits);
                for (int32_t n : lengths) {
                    if (n > most) continue;
                    const SplitRange r = split_range(n, window, __builtin_ctz((unsigned)splits), part_least_log(units));
                    int32_t p = parts_of(units, r.count);
                    if (p > splits) p = splits;
                    const int32_t chunk = ((r.count + p - 1) / p + 127) / 128 * 128;
                    need(r.chunk == chunk, "chunk", c, most, n, window, r.chunk);
                    need(r.count <= 512 ? r.used() == 1 : (r.chunk >= 512 || (r.chunk >= 256 && units * (p / 2) < 256)), "short parts", c, most, n, window,
                         r.chunk);
                    // the same as in a call with no room for more
                    const int32_t own = split_count(c.sequences, c.heads, c.kv_heads, n, window);
                    const SplitRange s = split_range(n, window, __builtin_ctz((unsigned)own), part_least_log(units));
                    need(s.chunk == r.chunk && s.used() == r.used(), "another max_length", c, most, n, window, r.chunk);
                }
            }
    }
    std::puts("ok");
}
"""


def test_parts_go_by_the_sequence(tmp_path):
    (tmp_path / "p.cpp").write_text(SOURCE)
    exe = str(tmp_path / "p")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", CSRC, str(tmp_path / "p.cpp"),
                           "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr[-2000:]
