"""Which kernel sizes choose for the block-scaled products (csrc/gemm_block_choice.h, compiled here
for the host): the sizes of test_gpu_layer_formats.py reach each of them, and the boundaries lie
where the rule's comment says."""
import os
import re
import subprocess

import pytest

from test_gpu_layer_formats import DENSE, EXPERTS

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_floating_point_amd", "csrc")
NAMES = re.findall(r"^\s+(k(?:Stream|Tile)\w+),", open(os.path.join(CSRC, "gemm_block_choice.h")).read(), re.M)


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("choice")
    (d / "c.cpp").write_text('#include "gemm_block_choice.h"\n#include <cstdio>\n#include <cstdlib>\nint main(int, char** v) {\n'
                             '    std::printf("%d", (int)fp4::block_kernel(std::atoi(v[1]), std::atoll(v[2]), std::atoll(v[3])));\n}\n')
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-I", CSRC, str(d / "c.cpp"), "-o", str(d / "c")])
    return lambda experts, M, N: NAMES[int(subprocess.check_output([str(d / "c"), str(experts), str(M), str(N)]))]


def test_every_kernel_is_tested(choose):
    assert set(DENSE) == set(EXPERTS) == set(NAMES) and len(NAMES) == 8
    for name, (M, N, _) in DENSE.items():
        assert choose(0, M, N) == name
    for name, (S, E, N, _) in EXPERTS.items():
        assert choose(E, S, N) == name


@pytest.mark.parametrize("experts,M,N,name", [
    (0, 1, 11008, "kStream64"), (0, 16, 4799, "kStream16"), (0, 16, 4800, "kStream32"), (0, 17, 4800, "kTile64K4"),
    (0, 64, 4096, "kTile64K4"), (0, 203, 4100, "kTile64K2"), (0, 1024, 4096, "kTile128K2"), (0, 2048, 4096, "kTile128"),
    (0, 4096, 15360, "kTile256"), (64, 64, 4096, "kStream64"), (64, 256, 4096, "kStream64"), (64, 512, 4096, "kTile128"),
    (64, 32768, 4096, "kTile256")])
def test_choice(choose, experts, M, N, name):
    assert choose(experts, M, N) == name
