"""Cases of the layer operators around the 8-bit floating-point products: the norm and SwiGLU
that write 8-bit activations with their scales, the product whose operands carry a scale per
block of 128, the routing of tokens to experts and the experts' products.

``own`` false: each operator in elementary torch operations, in binary32, rounded once at the
end.  ``own`` true: the calls of ``bit_floating_point_amd``.  Codes are returned as the values
they stand for (float8 tensors); their scales are outputs of their own.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-5


# ---------------------------------------------------------------- cases ---------------
def listed():
    return [
        # one decoded token of a 13B-shaped layer: residual stream, norm, codes with one scale per token
        {"name": "norm 1x5120 row", "op": "norm", "rows": 1, "cols": 5120, "terms": 1, "x": "bf16", "residual": "bf16",
         "grid": "e4m3", "gran": "row", "group": 0, "y": False, "static": False},
        # a calibrated (static) scale with pre-shifted channels, binary32 stream, odd row count and width
        {"name": "norm 777x11016 static", "op": "norm", "rows": 777, "cols": 11016, "terms": 1, "x": "f32",
         "residual": "f32", "grid": "e5m2", "gran": "tensor", "group": 0, "y": False, "static": True},
        # 4096 prefill tokens after an expert layer: eight weighted expert outputs join the residual,
        # the normalised rows are kept for the next router
        {"name": "norm 4096x5120 of 8 terms", "op": "norm", "rows": 4096, "cols": 5120, "terms": 8, "x": "bf16",
         "residual": "bf16", "grid": "e4m3", "gran": "group", "group": 128, "y": True, "static": False},
        # the eight expert rows of one decoded token
        {"name": "swiglu 8x2048", "op": "swiglu", "rows": 8, "cols": 2048, "x": "bf16", "grid": "e4m3", "gran": "group",
         "group": 128, "static": False},
        # the dense MLP of a 13B-shaped prefill
        {"name": "swiglu 4096x13824", "op": "swiglu", "rows": 4096, "cols": 13824, "x": "bf16", "grid": "e4m3",
         "gran": "group", "group": 128, "static": False},
        # one decoded token through a 7B-shaped up projection: bound by reading the weights
        {"name": "product 1x11008x4096", "op": "product", "M": 1, "N": 11008, "K": 4096, "a": "e4m3", "w": "e4m3"},
        # a short ragged batch: no size a multiple of a tile, the last blocks of N and K cut
        {"name": "product 203x4100x2080", "op": "product", "M": 203, "N": 4100, "K": 2080, "a": "e4m3", "w": "e4m3"},
        # the QKV projection of a 13B-shaped prefill
        {"name": "product 4096x15360x5120", "op": "product", "M": 4096, "N": 15360, "K": 5120, "a": "e4m3", "w": "e4m3"},
        # routing of one decoded token
        {"name": "route 1 of 64", "op": "route", "T": 1, "E": 64, "top_k": 6, "score": "softmax", "groups": 1,
         "top_groups": 1, "group_top": 1, "bias": False, "renorm": True, "logits": "f32"},
        # prefill routing with a balance bias, groups, padding tokens and unavailable experts
        {"name": "route 16384 of 256 grouped", "op": "route", "T": 16384, "E": 256, "top_k": 8, "score": "sigmoid",
         "groups": 8, "top_groups": 4, "group_top": 2, "bias": True, "renorm": True, "logits": "f32"},
        # gate and up products of the experts of eight decoded tokens
        {"name": "experts 8 tokens", "op": "experts", "T": 8, "E": 64, "top_k": 8, "N": 4096, "K": 5120, "shared_rows": True},
        # the same products over 4096 prefill tokens
        {"name": "experts 4096 tokens", "op": "experts", "T": 4096, "E": 64, "top_k": 8, "N": 4096, "K": 5120,
         "shared_rows": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _granularity(rng):
    gran, group = rng.choice([("row", 0), ("group", 128), ("group", 128), ("group", 64), ("tensor", 0)])
    return {"gran": gran, "group": group, "static": gran == "tensor"}


def draw(rng):
    op = rng.choice(["norm", "swiglu", "product", "route", "experts"])
    if op == "norm":
        terms = rng.choice([1, 1, 2, 6, 8])
        cols = 8 * _log(rng, 32, 1728)
        rows = _log(rng, 1, min(8192, 4096 * 5120 * 8 // (cols * terms)))
        return {"op": op, "rows": rows, "cols": cols, "terms": terms, "x": rng.choice(["bf16", "f32"]) if terms == 1 else "bf16",
                "residual": rng.choice(["bf16", "f32", "none"]), "grid": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "y": rng.random() < 0.5, **_granularity(rng)}
    if op == "swiglu":
        cols = 8 * _log(rng, 16, 1728)
        rows = _log(rng, 1, min(32768, 4096 * 13824 // cols))
        return {"op": op, "rows": rows, "cols": cols, "x": rng.choice(["bf16", "bf16", "f32"]) if rows * cols < 2048 * 13824 else "bf16",
                "grid": rng.choice(["e4m3", "e4m3", "e5m2"]), **_granularity(rng)}
    if op == "product":
        N, K = _log(rng, 64, 15360), 16 * _log(rng, 8, 864)
        M = _log(rng, 1, min(4096, 4096 * 15360 * 5120 // (N * K)))
        a, w = rng.choice([("e4m3", "e4m3"), ("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
        return {"op": op, "M": M, "N": N, "K": K, "a": a, "w": w}
    if op == "route":
        E, groups, top_groups = rng.choice([(8, 1, 1), (16, 1, 1), (60, 1, 1), (64, 1, 1), (64, 8, 3), (160, 8, 3), (160, 1, 1),
                                            (256, 8, 4), (256, 1, 1), (384, 1, 1)])
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "top_k": rng.choice([1, 2, 4, 6, 8]), "score": score, "groups": groups,
                "top_groups": top_groups, "group_top": rng.choice([1, 2]), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.7,
                "logits": rng.choice(["f32", "bf16"])}
    E, top_k = rng.choice([(8, 2), (16, 2), (60, 4), (64, 6), (64, 8), (128, 8)])
    N, K = _log(rng, 128, 4096), 16 * _log(rng, 8, 320)
    if E * N * K > 64 * 4096 * 5120:
        N //= 2
    return {"op": op, "T": _log(rng, 1, 4096), "E": E, "top_k": top_k, "N": N, "K": K, "shared_rows": rng.random() < 0.5}


def _units(case):
    rows, cols = case["rows"], case["cols"]
    return 0 if case["gran"] == "tensor" else rows if case["gran"] == "row" else rows * -(-cols // case["group"])


def _experts_hit(case):
    """Expected number of experts that some token chooses (even popularity)."""
    return case["E"] * (1 - (1 - case["top_k"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    if op == "norm":
        rows, cols, n = case["rows"], case["cols"], case["rows"] * case["cols"]
        size = {"bf16": 2, "f32": 4, "none": 0}
        per = case["terms"] * size[case["x"]] + 2 * size[case["residual"]] + 1 + (2 if case["y"] else 0)
        extra = cols * (2 + (1 if case["static"] else 0)) + 4 * _units(case) + (4 * rows * case["terms"] if case["terms"] > 1 else 0)
        return {"bytes": n * per + extra, "flops": n * (2 * case["terms"] + 7)}
    if op == "swiglu":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (2 * (2 if case["x"] == "bf16" else 4) + 1) + 4 * _units(case), "flops": 8 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": M * K + N * K + 2 * M * N + 4 * (M * kb + nb * kb), "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        return {"bytes": T * E * (4 if case["logits"] == "f32" else 2) + 12 * T * k + 4 * (E + 1) + (4 * E if case["bias"] else 0),
                "flops": T * E * 8}
    T, E, k, N, K = (case[v] for v in ("T", "E", "top_k", "N", "K"))
    kb, nb, rows = -(-K // BLOCK), -(-N // BLOCK), T * (1 if case["shared_rows"] else k)
    return {"bytes": rows * (K + 4 * kb) + _experts_hit(case) * (N * K + 4 * nb * kb) + 2 * T * k * N + 4 * T * k + 4 * (E + 1),
            "flops": 2 * T * k * N * K}


# ---------------------------------------------------------------- inputs --------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _rand(g, *shape):
    return torch.rand(*shape, device=DEV, generator=g)


def _activations(g, rows, cols):
    """N(0, 1) tokens with 1% of the channels 50 times larger."""
    x = _randn(g, rows, cols)
    x *= torch.where(_rand(g, cols) < 0.01, 50.0, 1.0)
    return x


def _row_blocks(x, grid):
    """Codes [rows, K] and a scale per row and 128 columns."""
    rows, K = x.shape
    kb = -(-K // BLOCK)
    v = torch.nn.functional.pad(x, (0, kb * BLOCK - K)).view(rows, kb, BLOCK)
    s = v.abs().amax(2) / QMAX[grid]
    q = (v / s.clamp_min(1e-30)[:, :, None]).clamp(-QMAX[grid], QMAX[grid]).view(rows, kb * BLOCK)[:, :K]
    return q.to(FLOAT8[grid]).contiguous(), s


def _square_blocks(w, grid):
    """Codes [..., N, K] and a scale per 128 rows and 128 columns."""
    N, K = w.shape[-2:]
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    v = torch.nn.functional.pad(w, (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(-1, nb, BLOCK, kb, BLOCK)
    s = v.abs().amax((2, 4)) / QMAX[grid]
    q = (v / s.clamp_min(1e-30)[:, :, None, :, None]).clamp(-QMAX[grid], QMAX[grid])
    q = q.view(-1, nb * BLOCK, kb * BLOCK)[:, :N, :K].to(FLOAT8[grid])
    return q.reshape(w.shape).contiguous(), s.reshape(w.shape[:-2] + (nb, kb))


def _code_buffers(case, rows, cols):
    codes = torch.zeros(rows, cols, dtype=torch.uint8, device=DEV)
    scales = None if case["gran"] == "tensor" else torch.zeros(_units(case), device=DEV)
    return {"codes": codes, "values": codes.view(FLOAT8[case["grid"]]), "scales": scales}


def _prepare_norm(case, g):
    rows, cols, terms = case["rows"], case["cols"], case["terms"]
    st = {"x": _activations(g, rows * terms, cols).to(DTYPES[case["x"]]), "gamma": (1 + 0.1 * _randn(g, cols)).bfloat16(),
          "weights": None, "residual": None, "residual_out": None, "y": None, "scale": None, "shift": None}
    if terms > 1:
        w = torch.softmax(_randn(g, rows, terms), 1)
        gone = _rand(g, rows, terms) < 0.02  # slots without an expert: weight 0 over a row that nothing wrote
        st["weights"] = w.masked_fill(gone, 0.0)
        st["x"].view(rows, terms, cols).masked_fill_(gone[:, :, None], float("nan"))
    if case["residual"] != "none":
        st["residual"] = (3 * _activations(g, rows, cols)).to(DTYPES[case["residual"]])
        st["residual_out"] = torch.zeros_like(st["residual"])
    if case["y"]:
        st["y"] = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    if case["static"]:
        st["scale"] = torch.full((1,), 4.0 / QMAX[case["grid"]], device=DEV)
        st["shift"] = -torch.randint(0, 4, (cols,), device=DEV, generator=g).to(torch.int8)
    return {**st, **_code_buffers(case, rows, cols)}


def _prepare_swiglu(case, g):
    rows, cols = case["rows"], case["cols"]
    st = {"x": (2 * _randn(g, rows, 2 * cols)).to(DTYPES[case["x"]]), "scale": None, "shift": None}
    if case["static"]:
        st["scale"] = torch.full((1,), 8.0 / QMAX[case["grid"]], device=DEV)
        st["shift"] = -torch.randint(0, 4, (cols,), device=DEV, generator=g).to(torch.int8)
    return {**st, **_code_buffers(case, rows, cols)}


def _prepare_product(case, g):
    M, N, K = case["M"], case["N"], case["K"]
    a, sa = _row_blocks(_activations(g, M, K), case["a"])
    w, sw = _square_blocks(0.02 * _randn(g, N, K), case["w"])
    return {"a": a, "sa": sa, "w": w, "sw": sw, "a_codes": a.view(torch.uint8), "w_codes": w.view(torch.uint8),
            "y": torch.zeros(M, N, dtype=torch.bfloat16, device=DEV)}


def _logits(case, g):
    """Router logits.  Which of two experts wins where their keys agree in all but the last bits of
    binary32 is a matter of rounding: tokens whose choice hangs on that get another token's logits."""
    T, E, k = case["T"], case["E"], case["top_k"]
    n = T + 64
    logits = (_randn(g, n, E) + 0.5 * _randn(g, E)).bfloat16()
    bias = (0.1 * _randn(g, E)) if case["bias"] else None
    if T > 1:
        logits[_rand(g, n, E) < 0.01] = -math.inf  # experts that a token may not use
        logits[:T][_rand(g, T) < 0.01] = -math.inf  # padding tokens
    key = _exact_scores(case, logits.double())
    key = torch.where(torch.isfinite(logits), key + (bias.double() if bias is not None else 0.0), -math.inf)
    group, kept = _exact_groups(case, key)

    def hangs(v, count):  # a gap among the first `count` + 1 in order that rounding could turn round
        v = v.sort(dim=1, descending=True).values[:, :count + 1]
        return ((v[:, :-1] - v[:, 1:]).nan_to_num(1.0, 1.0, 1.0) < 1e-6).any(1) if v.shape[1] > 1 else torch.zeros(len(v), dtype=torch.bool, device=DEV)

    same = hangs(kept, k) | (hangs(group, case["top_groups"]) if case["groups"] > 1 else False)
    good = torch.nonzero(~same).view(-1)
    pick = torch.where(same, good[torch.randint(0, len(good), (n,), device=DEV, generator=g)], torch.arange(n, device=DEV))[:T]
    return logits[pick].to(DTYPES[case["logits"]]).contiguous(), bias


def _prepare_route(case, g):
    T, E, k = case["T"], case["E"], case["top_k"]
    logits, bias = _logits(case, g)
    ints = {"dtype": torch.int32, "device": DEV}
    return {"logits": logits, "bias": bias, "experts": torch.zeros(T, k, **ints), "weights": torch.zeros(T, k, device=DEV),
            "offsets": torch.zeros(E + 1, **ints), "slots": torch.zeros(T * k, **ints)}


def _prepare_experts(case, g):
    T, E, k, N, K = (case[v] for v in ("T", "E", "top_k", "N", "K"))
    rows = T if case["shared_rows"] else T * k
    a, sa = _row_blocks(_activations(g, rows, K), "e4m3")
    w, sw = _square_blocks(0.02 * _randn(g, E, N, K), "e4m3")
    popular = _randn(g, T, E) + 0.5 * _randn(g, E)
    chosen = popular.argsort(dim=1, descending=True, stable=True)[:, :k]
    if T > 8:
        chosen = torch.where(_rand(g, T, 1) < 0.01, E, chosen)  # padding tokens: no expert
    flat = chosen.reshape(-1)
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return {"a": a, "sa": sa, "w": w, "sw": sw, "a_codes": a.view(torch.uint8), "w_codes": w.view(torch.uint8),
            "offsets": offsets, "slots": flat.argsort(dim=0, stable=True).to(torch.int32),
            "y": torch.zeros(T * k, N, dtype=torch.bfloat16, device=DEV)}


def prepare(case, seed):
    make = {"norm": _prepare_norm, "swiglu": _prepare_swiglu, "product": _prepare_product, "route": _prepare_route,
            "experts": _prepare_experts}
    return {"case": case, **make[case["op"]](case, _generator(seed))}


# ---------------------------------------------------------------- plain forms ---------
def _plain_codes(st, v):
    """Codes of v on the case's grid, and the scales of its units."""
    case, (rows, cols), qmax = st["case"], v.shape, QMAX[st["case"]["grid"]]
    if case["gran"] == "tensor":
        r = (1.0 / st["scale"]) * torch.exp2(-st["shift"].float())
        return [(v * r).clamp(-qmax, qmax).to(FLOAT8[case["grid"]])]
    width = cols if case["gran"] == "row" else case["group"]
    units = -(-cols // width)
    u = torch.nn.functional.pad(v, (0, units * width - cols)).view(rows, units, width)
    s = u.abs().amax(2) / qmax
    r = torch.where(s == 0, 0.0, 1.0 / s)
    q = (u * r[:, :, None]).clamp(-qmax, qmax).view(rows, units * width)[:, :cols]
    return [q.to(FLOAT8[case["grid"]]), s.view(-1)]


def _plain_norm(st):
    case = st["case"]
    rows, cols, terms = case["rows"], case["cols"], case["terms"]
    h = st["x"].float().view(rows, terms, cols)
    if st["weights"] is not None:
        w = st["weights"][:, :, None]
        h = torch.where(w == 0, 0.0, w * h)
    h = h.sum(1)
    if st["residual"] is not None:
        h = st["residual"].float() + h
    n = h * torch.rsqrt((h * h).sum(1, keepdim=True) / cols + EPS) * st["gamma"].float()
    out = _plain_codes(st, n)
    if st["residual"] is not None:
        out.append(h.to(st["residual"].dtype))
    if st["y"] is not None:
        out.append(n.bfloat16())
    return out


def _plain_swiglu(st):
    cols = st["case"]["cols"]
    gate, up = st["x"][:, :cols].float(), st["x"][:, cols:].float()
    return _plain_codes(st, gate / (1.0 + torch.exp(-gate)) * up)


def _spread(s, rows, cols, height):
    """A scale per block of `height` x 128, repeated over its block."""
    s = s.repeat_interleave(BLOCK, -1)[..., :cols]
    return s if height == 1 else s.repeat_interleave(height, -2)[..., :rows, :]


def _plain_product(st):
    a = st["a"].float() * _spread(st["sa"], *st["a"].shape, 1)
    w = st["w"].float() * _spread(st["sw"], *st["w"].shape, BLOCK)
    return [(a @ w.t()).bfloat16()]


def _plain_route(st):
    case, logits = st["case"], st["logits"].float()
    T, E, k, G = case["T"], case["E"], case["top_k"], case["groups"]
    usable = torch.isfinite(logits)
    if case["score"] == "softmax":
        top = torch.where(usable, logits, -math.inf).amax(1, keepdim=True)
        e = torch.where(usable, torch.exp(logits - top), 0.0)
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-logits))
    score = torch.where(usable, score, 0.0)
    key = torch.where(usable, score if st["bias"] is None else score + st["bias"], -math.inf)
    if G > 1:
        best = key.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :case["group_top"]]
        total = torch.where(best[:, :, :1] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(2, keepdim=True))
        order = total[:, :, 0].argsort(dim=1, descending=True, stable=True)
        inside = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        inside.scatter_(1, order[:, :case["top_groups"]], True)
        key = torch.where(inside.repeat_interleave(E // G, 1), key, -math.inf)
    value, index = key.sort(dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    none = value == -math.inf
    weight = torch.where(none, 0.0, score.gather(1, index))
    if case["renorm"]:
        total = weight.sum(1, keepdim=True)
        weight = torch.where(total > 0, weight / total, 0.0)
    flat = torch.where(none, E, index).view(-1)
    slots = flat.argsort(dim=0, stable=True)
    offsets = torch.searchsorted(flat[slots], torch.arange(E + 1, device=DEV))
    return [torch.where(none, -1, index).to(torch.int32), weight, offsets.to(torch.int32), slots.to(torch.int32)]


def _plain_experts(st):
    case = st["case"]
    T, E, k, N, K = (case[v] for v in ("T", "E", "top_k", "N", "K"))
    a = st["a"].float() * _spread(st["sa"], *st["a"].shape, 1)
    w = st["w"].float() * _spread(st["sw"], N, K, BLOCK)
    counts = st["offsets"][1:] - st["offsets"][:-1]
    rank = torch.arange(int(counts.max()), device=DEV)  # every expert's rows, padded to the longest list
    at = (st["offsets"][:-1, None] + rank).clamp_max(T * k - 1).long()
    slot = torch.where(rank < counts[:, None], st["slots"][at].long(), T * k)
    rows = a[(slot // k if case["shared_rows"] else slot).clamp_max(len(a) - 1)]
    y = torch.zeros(T * k + 1, N, device=DEV)
    y[slot.view(-1)] = torch.bmm(rows, w.transpose(1, 2).contiguous()).view(-1, N)
    return [y[:T * k].bfloat16()]


# ---------------------------------------------------------------- the calls -----------
@functools.lru_cache(None)
def _framework():
    """The package, and the grids and granularities that a program makes once."""
    import bit_floating_point_amd as F
    grids = {"e4m3": F.grid_minifloat(4, 3), "e5m2": F.grid_minifloat(5, 2)}
    grans = {(mode, group): F.gran(mode, group) for mode, group in (("row", 0), ("tensor", 0), ("group", 64), ("group", 128))}
    return F, grids, grans


def _call_norm(st):
    F, grids, grans = _framework()
    case = st["case"]
    F.fp4_rmsnorm_quant(st["x"], st["gamma"], grids[case["grid"]], grans[case["gran"], case["group"]], eps=EPS,
                        residual=st["residual"], residual_out=st["residual_out"], terms=case["terms"],
                        term_weights=st["weights"], tensor_scale=st["scale"], col_shift=st["shift"], y=st["y"],
                        packed=st["codes"], scales=st["scales"])
    return [v for v in (st["values"], st["scales"], st["residual_out"], st["y"]) if v is not None]


def _call_swiglu(st):
    F, grids, grans = _framework()
    case = st["case"]
    F.fp4_swiglu_quant(st["x"], grids[case["grid"]], grans[case["gran"], case["group"]], tensor_scale=st["scale"],
                       col_shift=st["shift"], packed=st["codes"], scales=st["scales"])
    return [v for v in (st["values"], st["scales"]) if v is not None]


def _call_product(st):
    F, grids, _ = _framework()
    case = st["case"]
    return [F.fp4_gemm_block(st["a_codes"], st["sa"], st["w_codes"], st["sw"], grids[case["a"]], grids[case["w"]], y=st["y"])]


def _call_route(st):
    F, _, _ = _framework()
    case = st["case"]
    F.fp4_route(st["logits"], case["top_k"], score=case["score"], bias=st["bias"], groups=case["groups"],
                top_groups=case["top_groups"], group_top=case["group_top"], renormalise=case["renorm"],
                experts=st["experts"], weights=st["weights"], offsets=st["offsets"], slots=st["slots"])
    return [st["experts"], st["weights"], st["offsets"], st["slots"]]


def _call_experts(st):
    F, grids, _ = _framework()
    case = st["case"]
    return [F.fp4_gemm_experts(st["a_codes"], st["sa"], st["w_codes"], st["sw"], grids["e4m3"], grids["e4m3"], st["offsets"],
                               st["slots"], slots_per_row=case["top_k"] if case["shared_rows"] else 1, y=st["y"])]


_PLAIN = {"norm": _plain_norm, "swiglu": _plain_swiglu, "product": _plain_product, "route": _plain_route, "experts": _plain_experts}
_CALLS = {"norm": _call_norm, "swiglu": _call_swiglu, "product": _call_product, "route": _call_route, "experts": _call_experts}


def run(state):
    return (_CALLS if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits -------------
def _exact_units(case, v, st):
    """v / scale before its rounding to a code (within the grid's range), and the scales."""
    rows, cols = v.shape
    top = QMAX[case["grid"]]
    if case["gran"] == "tensor":
        return [(v / st["scale"].double() / 2.0 ** st["shift"].double()).clamp(-top, top)]
    width = cols if case["gran"] == "row" else case["group"]
    parts = v.split(width, 1)
    peak = torch.stack([p.abs().amax(1) for p in parts], 1) / top
    return [torch.cat([p / peak[:, i:i + 1].clamp_min(1e-300) for i, p in enumerate(parts)], 1), peak.reshape(-1)]


def _exact_norm(case, st):
    rows, cols, terms = case["rows"], case["cols"], case["terms"]
    h = torch.zeros(rows, cols, dtype=torch.float64, device=DEV)
    for j in range(terms):
        x = st["x"][j::terms].double()
        if terms > 1:
            w = st["weights"][:, j:j + 1].double()
            x = torch.where(w != 0, x, torch.zeros_like(x)) * w
        h += x
    if st["residual"] is not None:
        h += st["residual"].double()
    n = h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * st["gamma"].double()
    return _exact_units(case, n, st) + ([h] if st["residual"] is not None else []) + ([n] if st["y"] is not None else [])


def _exact_swiglu(case, st):
    gate, up = st["x"].double().chunk(2, 1)
    return _exact_units(case, gate * torch.sigmoid(gate) * up, st)


def _exact_block_product(a, sa, w, sw):
    y = torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64, device=DEV)
    a, w = a.double(), w.double()
    for b, at in enumerate(range(0, a.shape[1], BLOCK)):
        left = a[:, at:at + BLOCK] * sa[:, b:b + 1].double()
        right = w[:, at:at + BLOCK] * sw[:, b].double().repeat_interleave(BLOCK)[:w.shape[0], None]
        y += left @ right.t()
    return y


def _exact_scores(case, logits):
    usable = torch.isfinite(logits)
    if case["score"] == "sigmoid":
        return torch.where(usable, torch.sigmoid(logits), 0.0)
    return torch.softmax(torch.where(usable, logits, -math.inf), 1).nan_to_num(0.0)


def _exact_groups(case, key):
    """The groups' totals, and the keys of the experts in the groups that are kept."""
    G = case["groups"]
    if G == 1:
        return None, key
    top = torch.topk(key.unflatten(1, (G, -1)), case["group_top"], dim=2).values
    total = torch.where(top > -math.inf, top, 0.0).sum(2).masked_fill(top[:, :, 0] == -math.inf, -math.inf)
    least = torch.topk(total, case["top_groups"], dim=1).values[:, -1:]
    return total, key.unflatten(1, (G, -1)).masked_fill((total < least)[:, :, None], -math.inf).flatten(1)


def _exact_route(case, st):
    logits, E, k = st["logits"].double(), case["E"], case["top_k"]
    score = _exact_scores(case, logits)
    key = score if st["bias"] is None else score + st["bias"].double()
    _, key = _exact_groups(case, torch.where(torch.isfinite(logits), key, -math.inf))
    value, index = (v[:, :k] for v in key.sort(dim=1, descending=True, stable=True))
    weight = score.gather(1, index).masked_fill(value == -math.inf, 0.0)
    if case["renorm"]:
        weight = (weight / weight.sum(1, keepdim=True)).nan_to_num(0.0)
    chosen = index.masked_fill(value == -math.inf, E)
    counts = torch.stack([(chosen == e).sum() for e in range(E)])
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return [chosen.masked_fill(chosen == E, -1), weight, offsets, torch.sort(chosen.flatten(), stable=True).indices]


def _exact_experts(case, st):
    k = case["top_k"]
    y = torch.zeros(case["T"] * k, case["N"], dtype=torch.float64, device=DEV)
    bounds = st["offsets"].tolist()
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi > lo:
            slot = st["slots"][lo:hi].long()
            row = slot // k if case["shared_rows"] else slot
            y[slot] = _exact_block_product(st["a"][row], st["sa"][row], st["w"][e], st["sw"][e])
    return [y]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "product":
        return [_exact_block_product(st["a"], st["sa"], st["w"], st["sw"])]
    return {"norm": _exact_norm, "swiglu": _exact_swiglu, "route": _exact_route, "experts": _exact_experts}[case["op"]](case, st)
