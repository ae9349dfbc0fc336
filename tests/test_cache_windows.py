"""The workspace of an attention with a window (csrc/attend_split.h), on the CPU: what a sequence sees is bounded by the
window and a tile, exactly, and the workspace of the largest max_length serves every smaller one."""
import os
import subprocess

import pytest

from bit_floating_point_amd import cache as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_floating_point_amd", "csrc")
WINDOWS = [1, 31, 32, 33, 480, 481, 482, 512, 700, 992, 993, 994, 2017, 4065, 1 << 20, (1 << 30) - 32, 1 << 30, 1 << 40, (1 << 63) - 1]

SOURCE = r"""
#include <cstdio>
#include <initializer_list>
#include <cstdlib>
#include "attend_split.h"
using namespace fp4;
int main() {
    for (int32_t window : {0, 1, 2, 31, 32, 33, 64, 481, 993, 2017}) {
        int64_t most = 0;  // positions of the longest range so far, over all lengths
        for (int32_t n = 0; n < 5000; n++) {
            const SplitRange r = split_range(n, window, 0, {});
            most = r.count > most ? r.count : most;
            if (most_seen(n, window) != most) {
                std::printf("window %d length %d: %lld seen, %lld said\n", window, n, (long long)most, (long long)most_seen(n, window));
                return 1;
            }
        }
    }
    std::puts("ok");
}
"""


def test_most_seen_is_what_is_seen(tmp_path):
    (tmp_path / "p.cpp").write_text(SOURCE)
    exe = str(tmp_path / "p")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I", CSRC, str(tmp_path / "p.cpp"),
                           "-o", exe])
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout + r.stderr[-2000:]


@pytest.mark.parametrize("window", WINDOWS)
@pytest.mark.parametrize("n,heads,kv_heads", [(1, 8, 8), (3, 40, 8), (17, 64, 1), (33, 15, 5), (300, 5, 5)])
def test_the_longest_workspace_serves_all(n, heads, kv_heads, window):
    """Never less for a longer max_length or a larger window."""
    size = C._call("fp4_attend_workspace_size")
    lengths = sorted({max(1, w + d) for w in WINDOWS if w <= 1 << 20 for d in range(-2, 36)} | {1 << e for e in range(10, 34)})
    last = 0
    for length in lengths:
        now = size(n, heads, kv_heads, 128, length, window)
        assert now >= last, (length, now, last)
        assert now <= size(n, heads, kv_heads, 128, length, 0)
        last = now
