"""examples/expert_layer.py: the layer operators together, at several shapes."""
import importlib.util
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m  # dataclasses look their module up
    spec.loader.exec_module(m)
    return m


# Activations enter twice as 3-bit mantissas (relative error uniform below 2^-4, at most
# 2^-4 / sqrt 3 = 0.036 in norm each) and three results are rounded to bf16 (2^-9): the parts
# add up in quadrature to 0.051 of the update, doubled here for what the products of gate and
# up make of it, plus the rounding of the stream itself (2^-9 of a stream that is at most a
# few times the update).
@pytest.mark.parametrize("tokens,width,inner,experts,top_k", [(1, 512, 256, 8, 2), (77, 528, 144, 12, 3), (600, 1024, 512, 16, 4)])
def test_layer(example, tokens, width, inner, experts, top_k):
    layer = example.make_layer(width, inner, experts, top_k, seed=tokens)
    g = torch.Generator(device="cuda")
    g.manual_seed(tokens)
    stream = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
    update = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
    err = example.relative_error(layer, stream, update)
    print(f"{err:.4f}", flush=True)
    assert err < 0.12
