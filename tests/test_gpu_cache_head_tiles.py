"""The attention with several tiles of query heads on a kv head, and over a cache of E4M3 with one given scale: scores that rise along the
sequence in some heads while they fall in others, so that each tile's running maximum moves at other positions, beside windows,
pages that are missing inside a sequence, and unseen rows of NaN.  Oracle and bounds are those of test_gpu_cache.py."""
import math

import pytest
import torch

import bit_floating_point_amd as F
from test_gpu_cache import DEV, DTYPES, check, gen, new_cache, reference, say

pytestmark = pytest.mark.gpu
I32 = torch.int32
FILL = {"bf16": 0xFF, "e4m3": 0x7F, "e5m2": 0x7F, "e2m1": 0xFF}  # NaN, in E2M1 -6 (its scales are NaN)
LENGTHS = [1500, 200, 33, 1, 0, 700]


def slopes(store, scales, dim, heads, seed):
    """A cache whose first column of keys rises or falls by 20 along every sequence; its table, with a page of the first and of the
    last sequence taken out, and everything that no sequence sees NaN."""
    size, g = 16, gen(seed)
    used = [-(-n // size) for n in LENGTHS]
    pages = sum(used) + 2
    cache = new_cache(store, scales, pages, heads, size, dim, "psh", FILL[store])
    order, at = torch.randperm(pages, generator=g).to(I32), 0
    table = torch.full((len(LENGTHS), max(used) + 1), 2 ** 31 - 1, dtype=I32)
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    table[0, 40], table[5, 0] = -1, pages
    tokens = [(b, t) for b, n in enumerate(LENGTHS) for t in range(n)]
    seq, pos = (torch.tensor(v, dtype=I32) for v in zip(*tokens))
    k, v = (torch.randn(len(tokens), heads, dim, generator=g) for _ in range(2))
    along = torch.tensor([20.0 * t / max(1, LENGTHS[b] - 1) - 10 for b, t in tokens])
    k[:, :, 0] = torch.where(seq % 2 == 0, along, -along)[:, None]
    table = table.to(DEV)
    F.fp4_cache_write(k.to(DEV), v.to(DEV), cache, table, pos.to(DEV), seq.to(DEV))
    return cache, table


def attend(cache, table, store, scales, dim, share, dtype, seed):
    """Heads below 16 take the slope as it is, the others turned round; every fourth far flatter."""
    heads = cache.kv_heads
    q = 0.2 * torch.randn(len(LENGTHS), heads, share, dim, generator=gen(seed))
    h = torch.arange(share)
    q[..., 0] = torch.where(h < 16, 4.0, -4.0) * torch.where(h % 4 == 3, 0.05, 1.0)
    q = q.view(len(LENGTHS), heads * share, dim).to(DTYPES[dtype]).to(DEV)
    n = torch.tensor(LENGTHS, dtype=I32, device=DEV)
    for window in (0, 300, 17):
        lse = torch.full((len(LENGTHS), heads * share), math.nan, device=DEV)
        y = F.fp4_attend(q, cache, table, n, scale=1.0, window=window, lse=lse)
        check(y, lse, reference(q, store, scales, cache, table, LENGTHS, 1.0, window, 1 << 30), dim, max(LENGTHS), dtype == "f32", y.dtype)
        assert bool((y[4] == 0).all()) and bool((lse[4] == -math.inf).all())
        assert torch.equal(y, F.fp4_attend(q, cache, table, n, scale=1.0, window=window, max_length=1500))


@pytest.mark.parametrize("share", [17, 20, 33])
@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("store,scales", [("bf16", "none"), ("e4m3", "f32"), ("e4m3", "f16"), ("e4m3", "given"), ("e5m2", "f32"), ("e5m2", "given"),
                                          ("e2m1", "f16"), ("e2m1", "given")])
def test_two_tiles(store, scales, dim, share):
    """bf16 q and y, rows of up to 128 values: a workgroup takes two tiles."""
    say("two tiles", store, scales, dim, share)
    cache, table = slopes(store, scales, dim, 2, 5)
    attend(cache, table, store, scales, dim, share, "bf16", 6)


@pytest.mark.parametrize("dim,share,dtype", [(64, 3, "bf16"), (64, 20, "f32"), (96, 1, "f32"), (96, 16, "bf16"), (128, 8, "bf16"), (128, 8, "f32"),
                                             (192, 5, "bf16"), (192, 20, "bf16"), (192, 4, "f32"), (256, 2, "bf16"), (256, 17, "f32")])
def test_e4m3_given(dim, share, dtype):
    """One given scale of keys and one of values."""
    say("e4m3 given", dim, share, dtype)
    cache, table = slopes("e4m3", "given", dim, 2, 7)
    attend(cache, table, "e4m3", "given", dim, share, dtype, 8)


def test_one_scale_for_both():
    """Keys and values may have the same given scale."""
    say("one scale for both")
    s = torch.full((1,), 0.02, device=DEV)
    cache = F.kv_cache(4, 2, 16, 64, F.grid_minifloat(4, 3), k_scale=s, v_scale=s)
    x = torch.randn(2, 40, 2, 64, generator=gen(9)).to(DEV)
    table, at = torch.tensor([[2, 0, 1]], dtype=I32, device=DEV), torch.arange(40, dtype=I32, device=DEV)
    F.fp4_cache_write(x[0], x[1], cache, table, at, torch.zeros_like(at))
    codes, _ = F.fp4_quantize_pack(x.view(-1, 64), F.grid_minifloat(4, 3), F.gran("tensor"), tensor_scale=s)
    for i, rows in enumerate((cache.k, cache.v)):
        got = rows[table[0].long()].transpose(1, 2).reshape(48, 2, 64)[:40]
        assert torch.equal(got, codes.view(2, 40, 2, 64)[i])
    q = torch.randn(1, 6, 64, generator=gen(10)).bfloat16().to(DEV)
    y = F.fp4_attend(q, cache, table, torch.tensor([40], dtype=I32, device=DEV))
    check(y, None, reference(q, "e4m3", "given", cache, table, [40], 0.125, 0, 48), 64, 40, False, y.dtype)
