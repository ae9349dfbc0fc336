"""Cases of the key/value cache operators: rows of keys and values quantized as they are written into
pages, read back, and the attention of one new token per sequence over such a cache.

``own`` false: each operator in elementary torch operations, in binary32, rounded once at the end.
``own`` true: the calls of ``bit_floating_point_amd``.  8-bit codes are returned as the values they
stand for (float8 tensors), packed 4-bit ones as the rows that are read back from them; scales are
outputs of their own.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
KEY_RANGE, VALUE_RANGE = 24.0, 5.0  # what calibrated (static) scales cover


# ---------------------------------------------------------------- cases ---------------
# store: what the cache holds; scales: one f32 or f16 per row (token and head), one given ("static"), or
# none (bf16).  page: positions in a page.  spread: "even" sequences are `length` long, "ragged" ones reach
# from nothing to `length`.
def listed():
    return [
        # the keys and values of eight decoded tokens
        {"name": "write 8 decoded e4m3", "op": "write", "tokens": 8, "seqs": 8, "start": 37, "pad": 0, "kv_heads": 8, "dim": 128,
         "page": 16, "store": "e4m3", "scales": "f32", "x": "bf16"},
        # a prompt batch of a 13B-shaped model: 40 heads, no shared ones
        {"name": "write 16384 prompt e4m3", "op": "write", "tokens": 16384, "seqs": 4, "start": 0, "pad": 0, "kv_heads": 40,
         "dim": 128, "page": 64, "store": "e4m3", "scales": "f32", "x": "bf16"},
        # a ragged chunk in the middle of three sequences, padded to a fixed batch, with calibrated scales
        {"name": "write 1003 static e5m2", "op": "write", "tokens": 1003, "seqs": 3, "start": 21, "pad": 40, "kv_heads": 5, "dim": 64,
         "page": 32, "store": "e5m2", "scales": "static", "x": "f32"},
        # a 4-bit cache written and read back: a prompt chunk whose attention runs on the values that the cache holds
        {"name": "write, read 4096 e2m1", "op": "round", "tokens": 4096, "seqs": 2, "start": 0, "pad": 0, "kv_heads": 32, "dim": 128,
         "page": 64, "store": "e2m1", "scales": "f16", "x": "bf16"},
        {"name": "write, read 77 e2m1", "op": "round", "tokens": 77, "seqs": 5, "start": 9, "pad": 3, "kv_heads": 3, "dim": 96,
         "page": 16, "store": "e2m1", "scales": "f32", "x": "f32"},
        # the context of a chunked prompt, read back for the next chunk's attention
        {"name": "read 2x6000 e4m3", "op": "read", "seqs": 2, "length": 6000, "spread": "even", "kv_heads": 40, "dim": 128, "page": 64,
         "store": "e4m3", "scales": "f32", "x": "bf16"},
        # a short one, in the widest heads
        {"name": "read 3x100 e5m2", "op": "read", "seqs": 3, "length": 100, "spread": "ragged", "kv_heads": 2, "dim": 256, "page": 16,
         "store": "e5m2", "scales": "f16", "x": "f32"},
        # one sequence of a 7B-shaped model, short: latency counts
        {"name": "attend 1x512 e4m3", "op": "attend", "seqs": 1, "length": 512, "spread": "even", "kv_heads": 32, "share": 1, "dim": 128,
         "page": 64, "store": "e4m3", "scales": "f32", "x": "bf16", "window": 0, "lse": False},
        # a serving batch of a 13B-shaped model
        {"name": "attend 16x4096 e4m3", "op": "attend", "seqs": 16, "length": 4096, "spread": "even", "kv_heads": 40, "share": 1,
         "dim": 128, "page": 64, "store": "e4m3", "scales": "f32", "x": "bf16", "window": 0, "lse": False},
        # many sequences with heads in groups of eight over a 4-bit cache, of all lengths
        {"name": "attend 96x8192 ragged e2m1", "op": "attend", "seqs": 96, "length": 8192, "spread": "ragged", "kv_heads": 8, "share": 8,
         "dim": 128, "page": 16, "store": "e2m1", "scales": "f16", "x": "bf16", "window": 0, "lse": False},
        # one very long document in an unquantized cache
        {"name": "attend 1x131072 bf16", "op": "attend", "seqs": 1, "length": 131072, "spread": "even", "kv_heads": 8, "share": 4,
         "dim": 128, "page": 128, "store": "bf16", "scales": "none", "x": "bf16", "window": 0, "lse": False},
        # sliding windows, calibrated scales, odd head counts and f32 outputs with their log-sums
        {"name": "attend 33x2999 window e5m2", "op": "attend", "seqs": 33, "length": 2999, "spread": "ragged", "kv_heads": 5, "share": 3,
         "dim": 64, "page": 32, "store": "e5m2", "scales": "static", "x": "f32", "window": 1000, "lse": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cache(rng, stores):
    store = rng.choice(stores)
    scales = "none" if store == "bf16" else rng.choice(["f32", "f32", "f16", "static"])
    return {"dim": rng.choice([64, 96, 128, 128, 128, 192, 256]), "page": rng.choice([16, 32, 64, 128, 256]), "store": store, "scales": scales,
            "x": rng.choice(["bf16", "bf16", "f32"])}


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read", "round"])
    if op == "attend":
        case = _cache(rng, ["bf16", "e4m3", "e4m3", "e5m2", "e2m1"])
        kv_heads, share = rng.choice([(1, 8), (2, 16), (4, 7), (5, 3), (8, 4), (8, 8), (16, 2), (32, 1), (40, 1), (3, 20)])
        most = (300_000_000 if case["store"] != "bf16" else 150_000_000) // (kv_heads * case["dim"])  # positions in all
        length = _log(rng, 1, min(131072, most))
        return {"op": op, "seqs": _log(rng, 1, max(1, min(256, most // length))), "length": length, "spread": rng.choice(["even", "ragged"]),
                "kv_heads": kv_heads, "share": share, **case, "window": rng.choice([0, 0, 0, 1 + length // 3]), "lse": rng.random() < 0.3}
    case = _cache(rng, ["e2m1"] if op == "round" else ["bf16", "e4m3", "e4m3", "e5m2"] + (["e2m1"] if op == "read" else []))
    kv_heads = rng.choice([1, 2, 5, 8, 16, 32, 40])
    tokens = _log(rng, 1, min(16384, 70_000_000 // (kv_heads * case["dim"])))
    if op == "read":
        seqs = _log(rng, 1, min(64, tokens))
        return {"op": op, "seqs": seqs, "length": max(1, tokens // seqs), "spread": rng.choice(["even", "ragged"]), "kv_heads": kv_heads, **case}
    seqs = tokens if rng.random() < 0.3 and tokens <= 256 else _log(rng, 1, min(16, tokens))
    return {"op": op, "tokens": tokens, "seqs": seqs, "start": rng.choice([0, 0, rng.randint(1, 200)]), "pad": rng.choice([0, 0, tokens // 9]),
            "kv_heads": kv_heads, **case}


def _lengths(case):
    n, length = case["seqs"], case["length"]
    if case["spread"] == "even":
        return [length] * n
    return [0 if i == 0 and n > 2 else (i * 7919 % n + 1) * length // n for i in range(n)]  # the first of three or more: empty


def _write_lengths(case):
    """New tokens of every sequence."""
    n, tokens = case["seqs"], case["tokens"] - case["pad"]
    return [tokens // n + (i < tokens % n) for i in range(n)]


def _row_bytes(case):
    return case["dim"] * {"bf16": 4, "e4m3": 2, "e5m2": 2, "e2m1": 1}[case["store"]] // 2


def _scale_bytes(case):
    return {"f32": 4, "f16": 2, "static": 0, "none": 0}[case["scales"]]


def work(case):
    size, row = 4 if case["x"] == "f32" else 2, 2 * case["kv_heads"] * (_row_bytes(case) + _scale_bytes(case))
    rows = 2 * case["kv_heads"] * case["dim"]  # values of a position's keys and values
    if case["op"] in ("write", "round"):
        n = case["tokens"] - case["pad"]
        both = case["op"] == "round"
        return {"bytes": n * (rows * size + row) * (2 if both else 1) + (12 if both else 8) * case["tokens"], "flops": (5 if both else 3) * n * rows}
    if case["op"] == "read":
        n = sum(_lengths(case))
        return {"bytes": n * (rows * size + row + 8), "flops": n * rows}
    seen = sum(min(n, case["window"] or n) for n in _lengths(case))
    heads, n = case["kv_heads"] * case["share"], case["seqs"]
    return {"bytes": seen * row + 2 * n * heads * case["dim"] * size + 4 * n + 4 * seen // case["page"] + (4 * n * heads if case["lse"] else 0),
            "flops": 4 * seen * heads * case["dim"]}


# ---------------------------------------------------------------- inputs --------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _keys(g, *shape):
    """Keys: N(0, 1) with two strong channels in every 64."""
    x = _randn(g, *shape)
    x *= torch.where(torch.rand(shape[-1], device=DEV, generator=g) < 0.03, 4.0, 1.0)
    return x


def _plain_rows(x, case, static):
    """What the cache holds of rows x (binary32), and their scales."""
    if case["store"] == "bf16":
        return x.bfloat16(), None
    qmax, s, kept = QMAX[case["store"]], static, None
    if s is None:
        s = x.abs().amax(-1, keepdim=True)
        s = s / torch.full_like(s, qmax)  # rounded once: a tensor over a number is its product with the reciprocal
        s = torch.where(s == 0, 0.0, s.clamp_min(2.0 ** -126))
        kept = s[..., 0].to(TYPES[case["scales"]])
        s = kept.float()[..., None]
    y = (x * torch.where(s == 0, 0.0, 1.0 / s)).clamp(-qmax, qmax)
    if case["store"] in FLOAT8:
        return y.to(FLOAT8[case["store"]]).view(torch.uint8), kept
    a, sign = y.abs(), torch.signbit(y).to(torch.uint8) * 8
    # the number of midpoints below the magnitude; on a midpoint the even code
    code = sum((a > m if i % 2 == 0 else a >= m).to(torch.uint8) for i, m in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0))) + sign
    return code[..., 0::2] + code[..., 1::2] * 16, kept


def _plain_values(codes, scales, case):
    """The rows that the cache's codes stand for, in binary32."""
    if case["store"] == "bf16":
        return codes.float()
    if case["store"] in FLOAT8:
        v = codes.view(FLOAT8[case["store"]]).float()
    else:
        grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
        v = torch.stack((grid[(codes & 15).int()], grid[(codes >> 4).int()]), -1).flatten(-2)
    return v * (scales if scales.numel() == 1 else scales.float()[..., None])


def _static(case):
    if case["scales"] != "static":
        return None, None
    return tuple(torch.full((1,), v / QMAX[case["store"]], device=DEV) for v in (KEY_RANGE, VALUE_RANGE))


def _pages(case, g, lengths):
    """A page table [seqs, pages of the longest] with pages in no order, -1 past a sequence's end."""
    counts = torch.tensor([-(-n // case["page"]) for n in lengths])
    total, most = int(counts.sum()), max(1, int(counts.max()))
    order = torch.randperm(total + 3, device=DEV, generator=g).to(torch.int32)
    used = torch.arange(most) < counts[:, None]
    place = torch.where(used, used.flatten().cumsum(0).view(used.shape) - 1, 0).to(DEV)
    return torch.where(used.to(DEV), order[place], -1).to(torch.int32), total + 3


def _prepare_cache(case, g, lengths):
    """A cache whose every slot holds a row: what is not used now is left of earlier sequences."""
    table, pages = _pages(case, g, lengths)
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    ks, vs = _static(case)
    k, k_scales = _plain_rows(_keys(g, *shape), case, ks)
    v, v_scales = _plain_rows(_randn(g, *shape), case, vs)
    return {"k_cache": k, "v_cache": v, "k_scales": ks if k_scales is None else k_scales, "v_scales": vs if v_scales is None else v_scales,
            "table": table}


def _prepare_write(case, g):
    counts = _write_lengths(case)
    st = _prepare_cache(case, g, [case["start"] + n for n in counts])
    sequences = [i for i, n in enumerate(counts) for _ in range(n)] + [0] * case["pad"]
    positions = [case["start"] + j for n in counts for j in range(n)] + [-1] * case["pad"]  # padding: no position
    # keys and values as they come out of one product: columns of wider rows
    heads, tokens = case["kv_heads"], case["tokens"]
    rows = torch.cat([_randn(g, tokens, heads, case["dim"]), _keys(g, tokens, heads, case["dim"]), _randn(g, tokens, heads, case["dim"])], 1)
    rows = rows.to(TYPES[case["x"]])
    st |= {"k": rows[:, heads:2 * heads], "v": rows[:, 2 * heads:], "positions": torch.tensor(positions, dtype=torch.int32, device=DEV),
           "sequences": torch.tensor(sequences, dtype=torch.int32, device=DEV) if sequences != list(range(len(sequences))) else None}
    if case["op"] == "round":
        st |= {"k_out": torch.zeros(tokens, heads, case["dim"], dtype=TYPES[case["x"]], device=DEV)}
        st |= {"v_out": torch.zeros_like(st["k_out"])}
    return st


def _prepare_read(case, g):
    lengths = _lengths(case)
    st = _prepare_cache(case, g, lengths)
    n = torch.tensor(lengths, device=DEV)
    st["sequences"] = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), n).to(torch.int32)
    first = n.cumsum(0) - n
    st["positions"] = (torch.arange(sum(lengths), device=DEV) - first[st["sequences"].long()]).to(torch.int32)
    st["k_out"] = torch.zeros(sum(lengths), case["kv_heads"], case["dim"], dtype=TYPES[case["x"]], device=DEV)
    return st | {"v_out": torch.zeros_like(st["k_out"])}


def _prepare_attend(case, g):
    lengths, heads = _lengths(case), case["kv_heads"] * case["share"]
    st = _prepare_cache(case, g, lengths)
    q = (1.5 * _randn(g, case["seqs"], heads, case["dim"])).to(TYPES[case["x"]])
    return st | {"q": q, "y": torch.zeros_like(q), "lengths": torch.tensor(lengths, dtype=torch.int32, device=DEV),
                 "lse": torch.zeros(case["seqs"], heads, device=DEV) if case["lse"] else None}


def prepare(case, seed):
    make = {"write": _prepare_write, "round": _prepare_write, "read": _prepare_read, "attend": _prepare_attend}[case["op"]]
    return {"case": case, **make(case, _generator(seed))}


# ---------------------------------------------------------------- plain forms ---------
def _held(st):
    """The cache as values of the types it holds, and its row scales."""
    case = st["case"]
    rows = [t.view(FLOAT8[case["store"]]) if case["store"] in FLOAT8 else t for t in (st["k_cache"], st["v_cache"])]
    return rows + ([st["k_scales"], st["v_scales"]] if _scale_bytes(case) else [])


def _places(st):
    """Page and slot of every token that has a position: padding comes last."""
    case = st["case"]
    n = case["tokens"] - case["pad"] if "tokens" in case else len(st["positions"])
    position = st["positions"][:n].long()
    sequence = torch.arange(n, device=DEV) if st["sequences"] is None else st["sequences"][:n].long()
    return n, st["table"][sequence, position // case["page"]].long(), position % case["page"]


def _plain_write(st):
    case = st["case"]
    n, page, slot = _places(st)
    static = (st["k_scales"], st["v_scales"]) if case["scales"] == "static" else (None, None)
    k, ks = _plain_rows(st["k"][:n].float(), case, static[0])
    v, vs = _plain_rows(st["v"][:n].float(), case, static[1])
    st["k_cache"][page, :, slot] = k
    st["v_cache"][page, :, slot] = v
    if ks is not None:
        st["k_scales"][page, :, slot] = ks
        st["v_scales"][page, :, slot] = vs
    return _held(st)


def _plain_read(st):
    case = st["case"]
    n, page, slot = _places(st)
    scales = (st["k_scales"], st["v_scales"])
    if _scale_bytes(case):
        scales = tuple(s[page, :, slot] for s in scales)
    k = _plain_values(st["k_cache"][page, :, slot], scales[0], case)
    v = _plain_values(st["v_cache"][page, :, slot], scales[1], case)
    gone = (0, 0, 0, 0, 0, len(st["positions"]) - n)  # padding reads as zeros
    return [torch.nn.functional.pad(t, gone).to(TYPES[case["x"]]) for t in (k, v)]


def _plain_round(st):
    _plain_write(st)
    return _plain_read(st) + ([st["k_scales"], st["v_scales"]] if _scale_bytes(st["case"]) else [])


def _plain_attend(st):
    case, n, dim = st["case"], st["case"]["seqs"], st["case"]["dim"]
    heads, share = case["kv_heads"], case["share"]
    pages = st["table"].clamp_min(0).long()

    def rows(cache, scales):  # [seqs, heads, positions, dim]
        if _scale_bytes(case):
            scales = scales[pages].transpose(1, 2).reshape(n, heads, -1)
        cache = cache[pages].transpose(1, 2)
        return _plain_values(cache.reshape(n, heads, -1, cache.shape[-1]), scales, case)
    k, v = rows(st["k_cache"], st["k_scales"]), rows(st["v_cache"], st["v_scales"])
    q = st["q"].float().view(n, heads, share, dim) * dim ** -0.5
    z = (k @ q.transpose(2, 3).contiguous()).transpose(2, 3)  # [seqs, heads, share, positions]
    at, length = torch.arange(k.shape[2], device=DEV), st["lengths"][:, None, None, None]
    seen = (at < length) & (at >= (length - case["window"] if case["window"] else 0))
    top = torch.where(seen, z, -math.inf).amax(3, keepdim=True)
    e = torch.where(seen, torch.exp(z - top), 0.0)
    total = e.sum(3, keepdim=True)
    y = (e.contiguous() @ v) * torch.where(total > 0, 1.0 / total, 0.0)
    out = [y.view(n, heads * share, dim).to(TYPES[case["x"]])]
    return out + [torch.where(total > 0, top + torch.log(total), -math.inf).view(n, heads * share)] if case["lse"] else out


# ---------------------------------------------------------------- the calls -----------
@functools.lru_cache(None)
def _framework():
    """The package, and the grids and granularities that a program makes once."""
    import bit_floating_point_amd as F
    grids = {"e4m3": F.grid_minifloat(4, 3), "e5m2": F.grid_minifloat(5, 2), "e2m1": F.grid_minifloat(2, 1), "bf16": None}
    grans = {"f32": F.gran("row"), "f16": F.gran("row", scale_dtype="f16"), "static": F.gran("tensor"), "none": None}
    return F, grids, grans


def _call(st):
    """The package, and the handle of the cache that a program makes once."""
    F, grids, grans = _framework()
    if "cache" not in st:
        case = st["case"]
        st["cache"] = F.KVCache(st["k_cache"], st["v_cache"], st["k_scales"], st["v_scales"], grids[case["store"]], grans[case["scales"]])
    return F, st["cache"]


def _call_write(st):
    F, cache = _call(st)
    F.fp4_cache_write(st["k"], st["v"], cache, st["table"], st["positions"], st["sequences"])
    return _held(st)


def _call_read(st):
    F, cache = _call(st)
    return list(F.fp4_cache_read(cache, st["table"], st["positions"], st["sequences"], k=st["k_out"], v=st["v_out"]))


def _call_round(st):
    F, cache = _call(st)
    F.fp4_cache_write(st["k"], st["v"], cache, st["table"], st["positions"], st["sequences"])
    read = F.fp4_cache_read(cache, st["table"], st["positions"], st["sequences"], k=st["k_out"], v=st["v_out"])
    return list(read) + ([st["k_scales"], st["v_scales"]] if _scale_bytes(st["case"]) else [])


def _call_attend(st):
    F, cache = _call(st)
    y = F.fp4_attend(st["q"], cache, st["table"], st["lengths"], window=st["case"]["window"], max_length=st["case"]["length"], y=st["y"],
                     lse=st["lse"])
    return [y] + ([st["lse"]] if st["lse"] is not None else [])


_PLAIN = {"write": _plain_write, "read": _plain_read, "round": _plain_round, "attend": _plain_attend}
_CALLS = {"write": _call_write, "read": _call_read, "round": _call_round, "attend": _call_attend}


def run(state):
    return (_CALLS if own else _PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- 64 bits -------------
def _exact_values(codes, scales, case):
    """The values of rows of codes, by the formulas of their formats; scales: one a row, or one."""
    if case["store"] == "bf16":
        return codes.double()
    if case["store"] in FLOAT8:
        v = codes.view(FLOAT8[case["store"]]).double()
    else:
        c = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
        power, half = c % 8 // 2, (c % 2).double() / 2
        v = torch.where(power == 0, half, (1 + half) * 2.0 ** (power - 1).double()) * (1 - 2 * (c // 8)).double()
    return v * (scales.double() if case["scales"] == "static" else scales.double().unsqueeze(-1))


def _exact_units(x, case, static):
    """x over its scale before the rounding to a code (within the grid's range), and the scales."""
    x = x.double()
    if case["store"] == "bf16":
        return x, None
    top = QMAX[case["store"]]
    peak = x.abs().amax(-1) / top if static is None else static.double()
    return (x / (peak.unsqueeze(-1).clamp_min(1e-300) if static is None else peak)).clamp(-top, top), None if static is not None else peak


def _exact_places(case, st):
    """Page and slot of the tokens that have a position (the first ones)."""
    live = st["positions"][st["positions"] >= 0].long()
    sequence = torch.arange(len(live), device=DEV) if st["sequences"] is None else st["sequences"][:len(live)].long()
    return st["table"].long()[sequence, live.div(case["page"], rounding_mode="floor")], live.remainder(case["page"])


def _exact_write(case, st):
    """The cache's rows before their rounding to codes (those that are not written: as they were)."""
    out, kept, (page, slot) = [], [], _exact_places(case, st)
    for x, cache, scales in ((st["k"], st["k_cache"], st["k_scales"]), (st["v"], st["v_cache"], st["v_scales"])):
        unit, peak = _exact_units(x[:len(page)], case, scales if case["scales"] == "static" else None)
        whole = (cache.view(FLOAT8[case["store"]]) if case["store"] in FLOAT8 else cache).double()
        whole[page, :, slot] = unit
        out.append(whole)
        if peak is not None:
            kept.append(scales.double())
            kept[-1][page, :, slot] = peak
    return out + kept


def _exact_round(case, st):
    """Rows written to a packed 4-bit cache and read back, and the scales.  Where a value lies between two codes is
    part of the definition, bit for bit: the scale, its reciprocal and their product are each rounded to binary32."""
    out, kept, (page, slot) = [], [], _exact_places(case, st)
    for x, scales in ((st["k"], st["k_scales"]), (st["v"], st["v_scales"])):
        rows = torch.zeros(x.shape, dtype=torch.float64, device=DEV)
        x = x[:len(page)].double()
        scale = scales.double()
        if case["scales"] != "static":
            peak = x.abs().amax(-1) / QMAX["e2m1"]
            kept.append(scale)
            kept[-1][page, :, slot] = peak
            scale = peak.float().to(scales.dtype).double().unsqueeze(-1)  # as it is held
        u = (x * (1 / torch.where(scale == 0, math.inf, scale)).float()).float().double().clamp(-QMAX["e2m1"], QMAX["e2m1"])
        step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0))  # between the grid's values
        rows[:len(page)] = torch.round(u / step) * step * scale
        out.append(rows)
    return out + kept


def _exact_sequence(case, st, b, lo, hi):
    """Keys and values of positions lo .. hi of a sequence: [kv_heads, positions, dim]."""
    first = lo // case["page"]
    page = st["table"][b, first:-(-hi // case["page"])].long()

    def positions(t):  # [pages, kv_heads, page, ..] -> [kv_heads, positions, ..]
        return torch.cat(list(t[page].unbind(0)), 1)[:, lo - first * case["page"]:hi - first * case["page"]]
    return [_exact_values(positions(cache), positions(scales) if _scale_bytes(case) else scales, case)
            for cache, scales in ((st["k_cache"], st["k_scales"]), (st["v_cache"], st["v_scales"]))]


def _exact_read(case, st):
    k, v = ([], [])
    for b, n in enumerate(_lengths(case)):
        if n:
            rows = _exact_sequence(case, st, b, 0, n)
            k.append(rows[0].transpose(0, 1))
            v.append(rows[1].transpose(0, 1))
    return [torch.cat(k), torch.cat(v)]


def _exact_attend(case, st):
    heads, share, dim = case["kv_heads"], case["share"], case["dim"]
    y = torch.zeros(case["seqs"], heads, share, dim, dtype=torch.float64, device=DEV)
    lse = torch.full((case["seqs"], heads, share), -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(_lengths(case)):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n > lo:
            k, v = _exact_sequence(case, st, b, lo, n)
            z = torch.bmm(st["q"][b].double().view(heads, share, dim), k.transpose(1, 2).contiguous()) / math.sqrt(dim)
            y[b], lse[b] = torch.bmm(torch.softmax(z, 2), v), torch.logsumexp(z, 2)
    out = [y.view(case["seqs"], heads * share, dim)]
    return out + [lse.view(case["seqs"], -1)] if case["lse"] else out


def exact(case, seed):
    make = {"write": _exact_write, "read": _exact_read, "round": _exact_round, "attend": _exact_attend}[case["op"]]
    return make(case, prepare(case, seed))
