"""examples/decode_attention.py: norm, products, cache and attention together, at several shapes, eagerly and as a
graph that is replayed while the sequences grow."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_attention.py")


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("decode_attention", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m  # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


# A value rounded to 3 bits of mantissa is off by at most 2^-4 of itself, uniformly: 0.036 in norm; E2M1 with a
# scale per row of 128 normal numbers: the largest is about 2.8 deviations, so that steps between codes are 0.23, 0.47 and
# 0.93 deviations and the error 0.07 .. 0.14, taken as 0.13.  The layer's output sees the rounding of its input (0.036 of
# v; and through q and k, as the scores are of order one and their error is relative in norm, 0.036 sqrt 2
# of the weights), of the cached v and k (c each) and of the output product's input (0.036).  In
# quadrature: sqrt(0.036^2 (1 + 2 + 1) + 2 c^2) = 0.072 (bf16: c = 0.001), 0.088 (E4M3), 0.20 (E2M1);
# doubled, for sequences of few positions, whose scores and errors do not average.
BOUNDS = {"bf16": 0.15, "e4m3": 0.18, "e2m1": 0.4}


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("width,heads,kv_heads,dim,size,prompts", [(256, 4, 4, 64, 16, [0, 1, 17]), (512, 8, 2, 128, 64, [100, 0, 900, 63]),
                                                                  (512, 6, 1, 256, 32, [1500])])
def test_steps(example, kind, width, heads, kv_heads, dim, size, prompts):
    layer = example.make_layer(width, heads, kv_heads, dim, seed=len(prompts))
    errors = example.relative_errors(layer, kind, prompts, 4, size)
    print(" ".join(f"{e:.4f}" for e in errors), flush=True)
    assert max(errors) < BOUNDS[kind]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_a_graph_of_the_step(example, kind):
    """Replays against the eager step on a cache of its own, bit for bit, other eager work and waits in between."""
    layer = example.make_layer(512, 8, 2, seed=3)
    both = [example.Pages(layer, 3, 2000, 64, kind) for _ in range(2)]
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    prompts = [1100, 0, 30]
    at = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompts]).cuda()
    of = torch.repeat_interleave(torch.arange(3, dtype=torch.int32), torch.tensor(prompts)).cuda()
    rows = torch.randn(sum(prompts), 512, device="cuda", generator=g).bfloat16()
    for pages in both:
        example.prompt(layer, pages, rows, of, at)
    x = torch.randn(3, 512, device="cuda", generator=g).bfloat16()
    for pages in both:
        example.step(layer, pages, x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = example.step(layer, both[0], x)
    for turn in range(6):
        x.copy_(torch.randn(3, 512, device="cuda", generator=g).bfloat16())
        if turn % 2:
            torch.cuda.synchronize()
        graph.replay()
        want = example.step(layer, both[1], x)
        assert torch.equal(y, want) and torch.equal(both[0].lengths, both[1].lengths)
        assert both[0].lengths.tolist() == [n + 2 + turn for n in prompts]
    assert torch.equal(both[0].cache.k, both[1].cache.k) and torch.equal(both[0].cache.v, both[1].cache.v)
