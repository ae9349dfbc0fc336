"""The attention over a cache at the ends of what include/fp4_cache.h allows: sums of values close to binary32's largest number
while the running maximum lags behind, and scores of 10^37."""
import math

import pytest
import torch

import bit_floating_point_amd as F
from test_gpu_cache import DEV, DTYPES, check, gen, new_cache, reference, say

pytestmark = pytest.mark.gpu
I32 = torch.int32
U = 2.0 ** -24


def stored(store, scales, k, v, size=16):
    """A cache of one sequence with these rows [positions, 1, dim], and its table."""
    n, _, dim = k.shape
    cache = new_cache(store, scales, -(-n // size), 1, size, dim)
    table = torch.arange(-(-n // size), dtype=I32, device=DEV)[None]
    at = torch.arange(n, dtype=I32, device=DEV)
    F.fp4_cache_write(k.to(DEV), v.to(DEV), cache, table, at, torch.zeros_like(at))
    return cache, table


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("store,scales", [("bf16", "none"), ("e4m3", "f32"), ("e5m2", "f32"), ("e2m1", "f32")])
@pytest.mark.parametrize("late", [0.0, 5.5])
def test_sums_at_the_bound(store, scales, dtype, late):
    """2^8 times the sum of 4096 values is 2^127.  With `late` 5.5 all positions after the first 128 have
    z log2 e = 7.93, which leaves the reference where it was: their weights are 2^7.93."""
    say("sums at the bound", store, dtype, late)
    n, dim, sequences = 4096, 64, 1024  # so many sequences that none is split
    k = torch.zeros(n, 1, dim)
    k[128:, 0, 0] = late
    v = (2.0 ** 107) * torch.where(torch.rand(n, 1, dim, generator=gen(1)) < 0.9, 1.0, -1.0)
    cache, table = stored(store, scales, k, v)
    q = torch.zeros(sequences, 1, dim)
    q[:, :, 0] = 1.0
    lengths = [n, n - 5, 200] + [0] * (sequences - 3)
    lse = torch.empty(sequences, 1, device=DEV)
    y = F.fp4_attend(q.to(DTYPES[dtype]).to(DEV), cache, table.expand(sequences, -1), torch.tensor(lengths, dtype=I32, device=DEV), scale=1.0,
                     lse=lse)
    ref = reference(q, store, scales, cache, table.expand(sequences, -1), lengths, 1.0, 0, n)
    check(y, lse, ref, dim, n, dtype == "f32", y.dtype)


@pytest.mark.parametrize("store,scales,size", [("bf16", "none", 9.5e37), ("e4m3", "f32", 1e35), ("e2m1", "f16", 1e36), ("e5m2", "given", 1e33)])
@pytest.mark.parametrize("sequences", [1, 1024])
def test_scores_at_the_bound(store, scales, size, sequences):
    """z is +-q by keys of +-1 and the halves of that; q is so large that q times the codes and log2 e just stays in binary32, and only
    positions of the largest z have weight.  (Which of them: z has a step of 10^30 there.)  Those hold one value, which y
    is but for roundings.  The reference rises from the lowest z to the highest, in one part (many sequences) and over several."""
    say("scores at the bound", store, sequences)
    n, dim = 1500, 64
    sign = torch.where(torch.rand(n, generator=gen(3)) < 0.1, 1.0, 0.5)
    sign[:300], sign[300:700] = -1.0, -0.5
    if scales == "given":
        sign *= 0.031 * 1024  # the given scale of keys times a code
    k = torch.zeros(n, 1, dim)
    k[:, 0, 0] = sign
    v = torch.randn(n, 1, dim, generator=gen(4))
    v[sign == sign.max()], v[sign == sign.min()] = v[0].clone(), v[1].clone()
    cache, table = stored(store, scales, k, v)
    q = torch.zeros(sequences, 2, dim)
    q[:, 0, 0], q[:, 1, 0] = size, -size
    lse = torch.empty(sequences, 2, device=DEV)
    lengths = [n] + [0] * (sequences - 1)
    y = F.fp4_attend(q.to(DEV), cache, table.expand(sequences, -1), torch.tensor(lengths, dtype=I32, device=DEV), scale=1.0, lse=lse)
    at = torch.arange(n, dtype=I32, device=DEV)
    kc, vc = (t[:, 0].double().cpu() for t in F.fp4_cache_read(cache, table, at, torch.zeros_like(at), dtype=torch.float32))
    for h, s in ((0, 1.0), (1, -1.0)):
        z = s * q[0, 0, 0].double() * kc[:, 0]
        top = z == z.max()
        want = vc[top][0]
        assert bool((vc[top] == want).all()) and int(top.sum()) > 50
        # sums of `n` terms (2 U a step on the matrix cores, U for the weights), weights as three terms, the quotient, joins, output
        tol = ((3 * (n + 64) + 32) * U + 2.0 ** -27) * want.abs()
        assert bool(((y[0, h].double().cpu() - want).abs() <= tol).all()), (h, (y[0, h].double().cpu() - want).abs().max())
        # the logarithm of the count is far below a rounding of z, whose factors round a few times
        assert lse[0, h].item() == pytest.approx(z.max().item(), rel=16 * U)
    assert bool((y[1:] == 0).all()) and bool((lse[1:] == -math.inf).all())
