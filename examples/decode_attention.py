"""An attention layer that decodes over an 8- or 4-bit key/value cache.

    python examples/decode_attention.py [--sequences 32] [--prompt 2000] [--steps 16] [--width 2048] [--heads 16] [--kv-heads 4] [--cache e4m3]

RMS norm -> products for queries, keys and values -> keys and values into the cache's pages -> attention of
the new tokens over their sequences -> output product.  Weights are quantized once, with a scale per
block of 128 x 128; activations carry a scale per token and 128 channels, cache rows one each.  Prompts go
through the same products and into the cache at once.  Prints the time of a step and how far its
output is from the same layer in 64 bits with keys and values that were never rounded.
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
CACHES = {"bf16": (None, None), "e4m3": (E4M3, F.gran("row")), "e2m1": (F.grid_minifloat(2, 1), F.gran("row", scale_dtype="f16"))}


@dataclass
class Layer:
    gamma: torch.Tensor       # [width]
    qkv: torch.Tensor         # codes [(heads + 2 kv_heads) dim, width] and their block scales
    qkv_scales: torch.Tensor
    out: torch.Tensor         # codes [width, heads dim]
    out_scales: torch.Tensor
    heads: int
    kv_heads: int
    dim: int


class Pages:
    """A cache and the pages that its sequences own, taken in any order."""

    def __init__(self, layer: Layer, sequences: int, most: int, size: int = 64, kind: str = "e4m3", seed: int = 0):
        each = -(-most // size)
        self.cache = F.kv_cache(sequences * each, layer.kv_heads, size, layer.dim, *CACHES[kind])
        g = torch.Generator()
        g.manual_seed(seed)
        self.table = torch.randperm(sequences * each, generator=g).to(torch.int32).view(sequences, each).cuda()
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device="cuda")


def make_layer(width: int, heads: int, kv_heads: int, dim: int = 128, seed: int = 0) -> Layer:
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale):
        return scale * torch.randn(*shape, device="cuda", generator=g)
    qkv, qkv_scales = F.fp4_quantize_block(normal((heads + 2 * kv_heads) * dim, width, scale=width ** -0.5), E4M3)
    out, out_scales = F.fp4_quantize_block(normal(width, heads * dim, scale=(heads * dim) ** -0.5), E4M3)
    return Layer(1 + normal(width, scale=0.1), qkv, qkv_scales, out, out_scales, heads, kv_heads, dim)


def project(layer: Layer, x: torch.Tensor):
    """Queries, keys and values [tokens, heads, dim] of rows x (bf16), as columns of one product."""
    a, a_scales = F.fp4_rmsnorm_quant(x, layer.gamma, E4M3, PER_128)
    y = F.fp4_gemm_block(a, a_scales, layer.qkv, layer.qkv_scales, E4M3, E4M3).view(len(x), -1, layer.dim)
    return y[:, :layer.heads], y[:, layer.heads:layer.heads + layer.kv_heads], y[:, layer.heads + layer.kv_heads:]


def prompt(layer: Layer, pages: Pages, x: torch.Tensor, sequences: torch.Tensor, positions: torch.Tensor) -> None:
    """Keys and values of the prompts' tokens, all sequences in one call."""
    _, k, v = project(layer, x)
    F.fp4_cache_write(k, v, pages.cache, pages.table, positions, sequences)
    pages.lengths.scatter_reduce_(0, sequences.long(), positions + 1, "amax")


def step(layer: Layer, pages: Pages, x: torch.Tensor) -> torch.Tensor:
    """One new token of every sequence.  Nothing here depends on the lengths on the host: a graph of it can be
    replayed while the sequences grow."""
    q, k, v = project(layer, x)
    F.fp4_cache_write(k, v, pages.cache, pages.table, pages.lengths)
    pages.lengths += 1
    y = F.fp4_attend(q, pages.cache, pages.table, pages.lengths)
    a, a_scales = F.fp4_quantize_pack(y.view(len(x), -1), E4M3, PER_128)
    return F.fp4_gemm_block(a, a_scales, layer.out, layer.out_scales, E4M3, E4M3)


def reference(layer: Layer, rows: list, x: torch.Tensor) -> torch.Tensor:
    """The step's output in 64 bits, on the same quantized weights: rows[b] are the tokens of sequence b so far."""
    def values(codes, scales):
        s = scales.double().repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :codes.shape[1]]
        return codes.view(torch.float8_e4m3fn).double() * s
    w, share, out = values(layer.qkv, layer.qkv_scales), layer.heads // layer.kv_heads, []
    for b, before in enumerate(rows):
        h = torch.cat([before, x[b:b + 1]]).double()
        h = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt() * layer.gamma.double()
        y = (h @ w.t()).view(len(h), -1, layer.dim).transpose(0, 1).contiguous()
        q, k, v = y[:layer.heads, -1:], y[layer.heads:layer.heads + layer.kv_heads], y[layer.heads + layer.kv_heads:]
        p = torch.softmax((q * k.repeat_interleave(share, 0)).sum(2) * layer.dim ** -0.5, 1)
        out.append((p[..., None] * v.repeat_interleave(share, 0)).sum(1).reshape(1, -1))
    return torch.cat(out) @ values(layer.out, layer.out_scales).t()


def relative_errors(layer: Layer, kind: str, prompts: list, steps: int, size: int = 64) -> list:
    """Norm of the error over the norm of the output, for every step after prompts of these lengths."""
    pages = Pages(layer, len(prompts), max(prompts) + steps, size, kind)
    width = layer.gamma.numel()
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rows = [torch.randn(n, width, device="cuda", generator=g).bfloat16() for n in prompts]
    at = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompts]).cuda()
    of = torch.repeat_interleave(torch.arange(len(prompts), dtype=torch.int32), torch.tensor(prompts)).cuda()
    if len(at):
        prompt(layer, pages, torch.cat(rows), of, at)
    errors = []
    for _ in range(steps):
        x = torch.randn(len(prompts), width, device="cuda", generator=g).bfloat16()
        got, want = step(layer, pages, x).double(), reference(layer, rows, x)
        errors.append(((got - want).norm() / want.norm()).item())
        rows = [torch.cat([r, x[b:b + 1]]) for b, r in enumerate(rows)]
    return errors


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("sequences", 32), ("prompt", 2000), ("steps", 16), ("width", 2048), ("heads", 16), ("kv-heads", 4)):
        p.add_argument("--" + name, type=int, default=value)
    p.add_argument("--cache", choices=list(CACHES), default="e4m3")
    a = p.parse_args()
    layer = make_layer(a.width, a.heads, a.kv_heads)
    errors = relative_errors(layer, a.cache, [100, 7, 300], 3)
    print(f"relative error of a step: {max(errors):.4f}")
    pages = Pages(layer, a.sequences, a.prompt + 3 * a.steps + 8, kind=a.cache)
    tokens = torch.randn(a.sequences * a.prompt, a.width, device="cuda").bfloat16()
    index = torch.arange(a.sequences * a.prompt, dtype=torch.int32, device="cuda")
    prompt(layer, pages, tokens, index // a.prompt, index % a.prompt)
    x = tokens[:a.sequences].contiguous()
    step(layer, pages, x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(layer, pages, x)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(2):  # the second time counts
        begin.record()
        for _ in range(a.steps):
            graph.replay()
        end.record()
        torch.cuda.synchronize()
    print(f"{a.sequences} sequences of {a.prompt} positions, {a.cache} cache: {begin.elapsed_time(end) / a.steps * 1e3:.0f} us a step")


if __name__ == "__main__":
    main()
