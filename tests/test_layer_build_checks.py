"""Checks on the compiled gfx950 code of the layer operators that need no GPU.

The tile kernel of the block-scaled products waits for its direct-to-LDS loads by count, so
its main loop may hold no other vector memory operation, and the number of loads between its
waits must be the one that the counts assume:
  * no kernel of the products or of the norm spills to scratch memory;
  * a direct-to-LDS load sits right after the M0 write of its own asm block;
  * every vector memory operation of the main loop is a direct-to-LDS load;
  * at the wait that opens the next stage, the loads issued since that stage's own are at
    least as many as the wait leaves in flight.
"""
import os
import re
import subprocess

import pytest

from bit_floating_point_amd import build as B

pytestmark = pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not installed")


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    d = tmp_path_factory.mktemp("asm")

    def one(src):
        out = d / (src + ".s")
        subprocess.run([B.HIPCC] + B.CFLAGS + ["--cuda-device-only", "-S", os.path.join(B.CSRC, src), "-o", str(out)],
                       check=True, capture_output=True)
        return out.read_text()
    return {src: one(src) for src in ("gemm_block.hip", "norm_quant.hip")}


def kernels(text, part):
    for name in re.findall(r"^(_Z\w*" + part + r"\w*):", text, re.M):
        i = text.index(name + ":")
        body = []
        for line in text[i:text.index(".Lfunc_end", i)].split("\n")[1:]:
            t = line.split(";")[0].strip()
            if t and (not t.startswith(".") or re.match(r"^\.LBB\w+:$", t)):
                body.append(t)
        yield name, body


LDS_LOAD = re.compile(r"^buffer_load_dword\S*\s.*\blds$")
VMEM = re.compile(r"^(buffer_|global_|flat_|scratch_)")


def main_loop(body):
    """The innermost loop that holds matrix instructions."""
    labels = {t[:-1]: i for i, t in enumerate(body) if t.endswith(":")}
    best = None
    for j, t in enumerate(body):
        m = re.match(r"^s_c?branch\S*\s+(\.LBB\w+)$", t)
        if m and labels.get(m.group(1), j) < j:
            loop = body[labels[m.group(1)]:j]
            if any("mfma" in u for u in loop) and (best is None or len(loop) < len(best)):
                best = loop
    return best


@pytest.mark.parametrize("src", ["gemm_block.hip", "norm_quant.hip"])
def test_no_scratch(asm, src):
    sizes = re.findall(r"\.private_segment_fixed_size:\s*(\d+)", asm[src])
    assert sizes and all(int(v) == 0 for v in sizes)


def test_loads_follow_their_m0(asm):
    seen = 0
    for name, body in kernels(asm["gemm_block.hip"], "block_gemm_tile_kernel"):
        for i, t in enumerate(body):
            if LDS_LOAD.match(t):
                assert body[i - 1].startswith("s_add_u32 m0, "), (name, body[i - 1])
                seen += 1
            elif re.search(r"\bm0\b", t):
                assert t.startswith("s_add_u32 m0, ") and LDS_LOAD.match(body[i + 1]), (name, t)
    assert seen


def test_main_loop_waits(asm):
    """Per step a wavefront issues LB + 1 loads (weights, scales) and LA loads (activations).
    The loop is walked as a ring of S steps' loads: at the barrier that opens stage b + 1 the
    loads of stage b + 1 are the oldest that may still be in flight."""
    found = 0
    for name, body in kernels(asm["gemm_block.hip"], "block_gemm_tile_kernel"):
        args = [int(v) for v in re.findall(r"Li(\d+)E", name)]
        _, _, bm, bn, wm, wn, stages, _ = args
        la, lb = bm * 128 // 1024 // (wm * wn), bn * 128 // 1024 // (wm * wn)
        group = la + lb + 1
        loop = main_loop(body)
        assert loop, name
        assert all(LDS_LOAD.match(t) for t in loop if VMEM.match(t)), name
        assert sum(bool(LDS_LOAD.match(t)) for t in loop) == group, name
        # loads issued in the step before each barrier, and what the barrier's wait leaves
        issued, waits = 0, []
        for i, t in enumerate(loop):
            if LDS_LOAD.match(t):
                issued += 1
            if t == "s_barrier":
                n = int(re.match(r"^s_waitcnt vmcnt\((\d+)\) lgkmcnt\(0\)$", loop[i - 1]).group(1))
                waits.append((issued, n))
        # the last barrier opens the next stage: after that stage's loads came those of the
        # S - 2 stages behind it and this step's so far
        before, left = waits[-1]
        assert left <= (stages - 2) * group + before, (name, waits)
        # an earlier one only separates the weights' readers from their next load: it waits for none
        assert all(n >= stages * group for _, n in waits[:-1]), (name, waits)
        found += 1
    assert found >= 8
