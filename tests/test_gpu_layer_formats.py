"""Block-scaled products and the experts' products: every pair of 8-bit formats on every kernel
that sizes choose, against 64 bits.  (Which kernel a size runs: test_layer_kernel_choice.py.)"""
import pytest
import torch

from test_gpu_layer import F, check_product, device_operand, device_scales, grid, product_reference, say

pytestmark = pytest.mark.gpu

DEV = "cuda"
PAIRS = [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")]

# kernel -> M, N, K
DENSE = {"kStream16": (3, 203, 400), "kStream32": (7, 5003, 1168), "kStream64": (14, 9701, 400), "kTile64K4": (70, 301, 1168),
         "kTile64K2": (203, 4100, 272), "kTile128K2": (1025, 2305, 400), "kTile128": (2049, 3601, 272), "kTile256": (1999, 8001, 1168)}
# kernel -> slots, experts, N, K
EXPERTS = {"kStream16": (8, 4, 301, 400), "kStream32": (16, 8, 700, 1168), "kStream64": (16, 8, 1301, 400), "kTile64K4": (90, 6, 301, 1168),
           "kTile64K2": (80, 8, 2501, 272), "kTile128K2": (800, 8, 2501, 400), "kTile128": (800, 8, 4203, 272),
           "kTile256": (4800, 8, 2501, 1168)}


@pytest.mark.parametrize("fa,fw", PAIRS)
@pytest.mark.parametrize("kernel", DENSE)
def test_product(kernel, fa, fw):
    M, N, K = DENSE[kernel]
    say("product", kernel, M, N, K, fa, fw)
    g = torch.Generator(device=DEV)
    g.manual_seed(M + N)
    a, av = device_operand(g, M, K, fa)
    w, wv = device_operand(g, N, K, fw)
    sa, sw = device_scales(g, M, -(-K // 128)), device_scales(g, -(-N // 128), -(-K // 128))
    ref, S = product_reference(av, sa, wv, sw)
    y = F.fp4_gemm_block(a, sa, w, sw, grid(fa), grid(fw), y_dtype=torch.float32)
    check_product(y, ref.cpu(), S.cpu(), K)
    for _ in range(2):
        assert torch.equal(F.fp4_gemm_block(a, sa, w, sw, grid(fa), grid(fw)), y.bfloat16())


@pytest.mark.parametrize("fa,fw", PAIRS)
@pytest.mark.parametrize("kernel", EXPERTS)
def test_experts(kernel, fa, fw):
    S, E, N, K = EXPERTS[kernel]
    say("experts", kernel, S, E, N, K, fa, fw)
    g = torch.Generator(device=DEV)
    g.manual_seed(S + N)
    a, av = device_operand(g, S, K, fa)
    w, wv = device_operand(g, N, K, fw, (E,))
    sa, sw = device_scales(g, S, -(-K // 128)), device_scales(g, E, -(-N // 128), -(-K // 128))
    # uneven lists, one without slots (of four or more), and slots without an expert
    weight = torch.rand(E, device=DEV, generator=g) + 0.2
    weight[1] = 0
    choice = torch.multinomial(weight, S, replacement=True, generator=g)
    choice[torch.rand(S, device=DEV, generator=g) < 0.02] = E
    slots = torch.sort(choice, stable=True).indices.int()
    offsets = torch.searchsorted(choice.sort().values, torch.arange(E + 1, device=DEV)).int()
    y = torch.full((S, N), 7.0, device=DEV)
    F.fp4_gemm_experts(a, sa, w, sw, grid(fa), grid(fw), offsets, slots, y=y)
    for e in range(E):
        s = torch.nonzero(choice == e).view(-1)
        if len(s):
            ref, mag = product_reference(av[s], sa[s], wv[e], sw[e])
            check_product(y[s], ref.cpu(), mag.cpu(), K)
    assert (y[choice == E] == 7).all()
    for _ in range(2):
        yb = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV)
        F.fp4_gemm_experts(a, sa, w, sw, grid(fa), grid(fw), offsets, slots, y=yb)
        assert torch.equal(yb, y.bfloat16())
