"""An expert MLP layer in 8-bit floating point, from residual stream to residual stream.

    python examples/expert_layer.py [--tokens 512] [--width 2048] [--inner 1024] [--experts 32] [--top-k 4]

RMS norm -> router -> gate/up products of the chosen experts -> SwiGLU -> down products -> the
experts' outputs join the residual stream (inside the next norm).  Weights are quantized once, with a
scale per block of 128 x 128; activations carry a scale per token and 128 channels.  Prints the time
of a layer and how far its update of the stream is from the same layer in 64 bits on the same
quantized weights.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_floating_point_amd as F  # noqa: E402

E4M3 = F.grid_minifloat(4, 3)
PER_128 = F.gran("group", 128)


@dataclass
class Layer:
    gamma: torch.Tensor       # [width]
    router: torch.Tensor      # [width, experts], f32
    bias: torch.Tensor        # [experts]: balances the choice, not the weights
    gate_up: torch.Tensor     # codes [experts, 2 inner, width] and their block scales
    gate_up_scales: torch.Tensor
    down: torch.Tensor        # codes [experts, width, inner]
    down_scales: torch.Tensor
    top_k: int


def make_layer(width: int, inner: int, experts: int, top_k: int, seed: int = 0, device: str = "cuda") -> Layer:
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def normal(*shape, scale):
        return scale * torch.randn(*shape, device=device, generator=g)
    gate_up, gate_up_scales = F.fp4_quantize_block(normal(experts, 2 * inner, width, scale=width ** -0.5), E4M3)
    down, down_scales = F.fp4_quantize_block(normal(experts, width, inner, scale=inner ** -0.5), E4M3)
    return Layer(1 + normal(width, scale=0.1), normal(width, experts, scale=width ** -0.5), normal(experts, scale=0.02),
                 gate_up, gate_up_scales, down, down_scales, top_k)


def forward(layer: Layer, stream: torch.Tensor, update: torch.Tensor):
    """One layer.  `update` (bf16 [tokens, width], an attention output say) joins `stream` (bf16,
    changed in place), the experts run on its norm, and their outputs come back as rows per token and
    expert with the weights that the next norm adds them with."""
    normed = torch.empty_like(stream)
    a, a_scales = F.fp4_rmsnorm_quant(update, layer.gamma, E4M3, PER_128, residual=stream, residual_out=stream, y=normed)
    logits = normed.float() @ layer.router
    route = F.fp4_route(logits, layer.top_k, score="sigmoid", bias=layer.bias)
    h = F.fp4_gemm_experts(a, a_scales, layer.gate_up, layer.gate_up_scales, E4M3, E4M3, route.offsets, route.slots,
                           slots_per_row=layer.top_k)
    h, h_scales = F.fp4_swiglu_quant(h, E4M3, PER_128)
    out = F.fp4_gemm_experts(h, h_scales, layer.down, layer.down_scales, E4M3, E4M3, route.offsets, route.slots)
    return out, route


def join(layer: Layer, stream: torch.Tensor, out: torch.Tensor, route) -> None:
    """The experts' outputs join the stream; a next layer does this in its own norm."""
    F.fp4_rmsnorm_quant(out, layer.gamma, residual=stream, residual_out=stream, terms=layer.top_k, term_weights=route.weights)


def reference(layer: Layer, stream: torch.Tensor, update: torch.Tensor, route) -> torch.Tensor:
    """The stream after the layer in 64 bits, with the same experts and quantized weights."""
    def values(codes, scales):
        s = scales.double().repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]
        return codes.view(torch.float8_e4m3fn).double() * s
    h = stream.double() + update.double()
    n = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * layer.gamma.double()
    score = torch.sigmoid(n @ layer.router.double())
    chosen = route.experts.long()
    weight = score.gather(1, chosen)
    weight = weight / weight.sum(1, keepdim=True)
    for e in range(layer.router.shape[1]):
        token, place = torch.nonzero(chosen == e, as_tuple=True)
        if len(token):
            gate, up = (n[token] @ values(layer.gate_up[e], layer.gate_up_scales[e]).t()).chunk(2, 1)
            y = (torch.nn.functional.silu(gate) * up) @ values(layer.down[e], layer.down_scales[e]).t()
            h.index_add_(0, token, weight[token, place][:, None] * y)
    return h


def relative_error(layer: Layer, stream: torch.Tensor, update: torch.Tensor) -> float:
    """Norm of the error over the norm of the layer's update of the stream."""
    got = stream.clone()
    out, route = forward(layer, got, update)
    join(layer, got, out, route)
    want = reference(layer, stream, update, route)
    return ((got.double() - want).norm() / (want - stream.double() - update.double()).norm()).item()


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 512), ("width", 2048), ("inner", 1024), ("experts", 32), ("top-k", 4)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    layer = make_layer(a.width, a.inner, a.experts, a.top_k)
    stream = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    update = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    print(f"relative error of the update: {relative_error(layer, stream, update):.4f}")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):  # the second time counts
        begin.record()
        for _ in range(20):
            out, route = forward(layer, stream, update)
        end.record()
        torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {a.experts} experts: {begin.elapsed_time(end) / 20 * 1e3:.0f} us a layer")


if __name__ == "__main__":
    main()
