"""Every main loop of the block-scaled products' tile kernels, in the compiled gfx950 code (no GPU
needed).

A kernel of the experts' products with tiles of 256 rows has two: one for full tiles, one for
tiles that are at most half full.  In each innermost loop that holds matrix instructions:
  * every vector memory operation is a direct-to-LDS load, and there are as many as a step's
    waits count;
  * the wait at the barrier that opens the next stage leaves no more loads in flight than were
    issued since that stage's own;
  * a barrier before it waits for no load that is still needed.
"""
import os
import re
import subprocess

import pytest

from bit_floating_point_amd import build as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")

LDS_LOAD = re.compile(r"^buffer_load_dword\S*\s.*\blds$")
VMEM = re.compile(r"^(buffer_|global_|flat_|scratch_)")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(tile and wavefront sizes, experts or not, instructions) of every tile kernel."""
    out = tmp_path_factory.mktemp("asm") / "gemm_block.s"
    subprocess.run([B.HIPCC] + B.CFLAGS + ["--cuda-device-only", "-S", os.path.join(B.CSRC, "gemm_block.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    text, found = out.read_text(), []
    for name in re.findall(r"^(_Z\w*block_gemm_tile_kernel\w*):", text, re.M):
        i = text.index("\n" + name + ":")
        lines = (line.split(";")[0].strip() for line in text[i + 1:text.index(".Lfunc_end", i)].split("\n")[1:])
        body = [t for t in lines if t and (not t.startswith(".") or re.match(r"^\.LBB\w+:$", t))]
        found.append(([int(v) for v in re.findall(r"Li(\d+)E", name)], "Lb1E" in name, body))
    return found


def main_loops(body):
    """The loops with matrix instructions that contain no smaller one."""
    labels = {t[:-1]: i for i, t in enumerate(body) if t.endswith(":")}
    spans = []
    for j, t in enumerate(body):
        m = re.match(r"^s_c?branch\S*\s+(\.LBB\w+)$", t)
        if m and labels.get(m.group(1), j) < j and any("mfma" in u for u in body[labels[m.group(1)]:j]):
            spans.append((labels[m.group(1)], j))
    return [body[a:b] for a, b in spans if not any((c, d) != (a, b) and a <= c and d <= b for c, d in spans)]


def check_loop(loop, sizes):
    _, _, bm, bn, wm, wn, stages, _ = sizes
    la, lb = bm * 128 // 1024 // (wm * wn), bn * 128 // 1024 // (wm * wn)
    group = la + lb + 1  # activations, weights, scales
    assert all(LDS_LOAD.match(t) for t in loop if VMEM.match(t)), "a vector memory operation that no wait counts"
    assert sum(bool(LDS_LOAD.match(t)) for t in loop) == group, "loads of a step"
    issued, waits = 0, []
    for i, t in enumerate(loop):
        if LDS_LOAD.match(t):
            issued += 1
        if t == "s_barrier":
            m = re.match(r"^s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$", loop[i - 1])
            assert m, "a barrier without its wait"
            waits.append((issued, int(m.group(1))))
    before, left = waits[-1]
    assert left <= (stages - 2) * group + before, "the next stage's loads may still be in flight"
    assert all(n >= stages * group for _, n in waits[:-1])
    return waits


def test_every_main_loop(kernels):
    assert len(kernels) >= 8
    for sizes, experts, body in kernels:
        loops = main_loops(body)
        bm, bn, wm, wn = sizes[2:6]
        full = bm // wm // 32 * (bn // wn // 32) * 2  # matrix instructions of a step
        counts = sorted(sum("mfma" in t for t in loop) for loop in loops)
        assert counts == ([full // 2, full] if experts and bm == 256 else [full]), (sizes, experts)
        for loop in loops:
            check_loop(loop, sizes)


def test_the_check_sees_mistakes(kernels):
    """On the text: an operation that no wait counts, and a wait that leaves one load too many, in
    each loop of each kernel."""
    for sizes, _, body in kernels:
        for loop in main_loops(body):
            with pytest.raises(AssertionError):
                check_loop(loop + ["global_load_dword v0, v[2:3], off"], sizes)
            last = max(i for i, t in enumerate(loop) if t == "s_barrier")
            n = int(re.search(r"vmcnt\((\d+)\)", loop[last - 1]).group(1))
            with pytest.raises(AssertionError):
                check_loop(loop[:last - 1] + [f"s_waitcnt vmcnt({n + 1}) lgkmcnt(0)"] + loop[last:], sizes)
