"""SwiGLU with a scale per row on every number of chunks per thread that its rule chooses: against
64 bits, and the same bits for any number of rows (a maximum has no order)."""
import pytest
import torch

from test_gpu_layer import F, U, check_codes, grid, randn, rng, say

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("rows,cols", [(1023, 2056), (1024, 2048), (1100, 2056), (1030, 8192), (1030, 8200), (1100, 32768),
                                       (20, 8200), (20, 16384), (20, 16392), (30, 32776), (1030, 32776)])
def test_swiglu_of_row_scales(rows, cols):
    say("swiglu", rows, cols)
    g = rng(rows + cols)
    x = 2 * randn(g, rows, 2 * cols)
    x[1] = 0
    x = x.bfloat16()
    p, s = F.fp4_swiglu_quant(x.to(DEV), grid("e4m3"), F.gran("row"))
    for at in (slice(0, 7), slice(rows - 5, rows)):
        q, t = F.fp4_swiglu_quant(x[at].to(DEV), grid("e4m3"), F.gran("row"))
        assert torch.equal(p[at], q) and torch.equal(s[at], t)
        gate, up = x[at].double().chunk(2, 1)
        h = gate / (1 + torch.exp(-gate)) * up
        check_codes("e4m3", q, t, h, (2 * gate.abs() + 8) * U * h.abs() + 2.0 ** -100 * up.abs(), "row")
    half = rows // 2
    q, t = F.fp4_swiglu_quant(x[half:].to(DEV), grid("e4m3"), F.gran("row"))
    assert torch.equal(p[half:], q) and torch.equal(s[half:], t)
