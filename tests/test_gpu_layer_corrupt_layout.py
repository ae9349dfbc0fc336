"""The experts' products on layouts that no routing writes: nothing outside the operands is touched,
and what is written is the product.  (Ranges that overlap hold more tiles than a launch has, so
some column blocks of a row may stay as they were.)"""
import pytest
import torch

from test_gpu_layer import F, grid, say

pytestmark = pytest.mark.gpu

DEV = "cuda"


def corrupt(slots, experts, K, N, offsets):
    """All experts alike, one row of activations: every slot's product is the same."""
    g = torch.Generator(device=DEV)
    g.manual_seed(slots)
    a = (torch.randn(1, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn)
    w = (torch.randn(N, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn)
    y = torch.full((slots + 1, N), 7.0, dtype=torch.bfloat16, device=DEV)
    kb, nb = -(-K // 128), -(-N // 128)
    F.fp4_gemm_experts(a.view(torch.uint8), torch.ones(1, kb, device=DEV), w.view(torch.uint8)[None].repeat(experts, 1, 1),
                       torch.ones(experts, nb, kb, device=DEV), grid("e4m3"), grid("e4m3"), offsets.int().to(DEV),
                       torch.arange(slots, dtype=torch.int32, device=DEV), slots_per_row=slots, y=y[:slots])
    one = F.fp4_gemm_block(a.view(torch.uint8), torch.ones(1, kb, device=DEV), w.view(torch.uint8), torch.ones(nb, kb, device=DEV),
                           grid("e4m3"), grid("e4m3"), y_dtype=torch.float32)
    # both within the bound of packed products of the exact value, one of them rounded to bf16
    S = a.double().abs() @ w.double().abs().t()
    bound = 2.0 ** -8 * one.abs() + (2 * ((2 * K + 2 * kb + 4) * 2.0 ** -24 + 7 * 2.0 ** -13) * 1.01 * S).float()
    close = (y[:slots].float() - one).abs() <= bound
    assert (close | (y[:slots] == 7)).all() and (y[slots] == 7).all()


@pytest.mark.parametrize("slots,experts", [(100, 16), (3000, 64), (40000, 8)])
def test_overlapping_ranges(slots, experts):
    """Every other expert has all slots."""
    say("overlapping", slots, experts)
    corrupt(slots, experts, 144, 300, torch.tensor([0, slots] * (experts // 2) + [0]))


@pytest.mark.parametrize("offsets", [[-5, 10 ** 9, -10 ** 9, 2 ** 31 - 1, -2 ** 31, 50, 20, 80, 90], [500] * 9, [0] * 8 + [2 ** 31 - 1],
                                     [2 ** 31 - 1, -2 ** 31] * 4 + [2 ** 31 - 1]])
def test_offsets_outside(offsets):
    say("offsets", offsets)
    corrupt(100, 8, 144, 300, torch.tensor(offsets))


def test_more_tiles_than_32_bits():
    """512 ranges of all 2^29 and some slots: over 2^31 tiles of 128 rows."""
    slots = (1 << 29) + 1000
    say("many tiles", slots)
    corrupt(slots, 1024, 16, 1, torch.tensor([0, slots] * 512 + [0]))
    torch.cuda.empty_cache()
