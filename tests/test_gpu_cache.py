"""The key/value cache against the CPU oracle and plain 64-bit forms: rows written as bf16 or codes and read
back (bit for bit), and the attention of one new token per sequence (within bounds counted from its
arithmetic), over types, head layouts, page sizes, lengths from nothing to many parts, windows, strides
and caches whose unused rows, scales and table entries hold anything."""
import math

import numpy as np
import pytest
import torch

import bit_floating_point_amd as F
import oracle as O

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24  # half a step of binary32
GRIDS = {"bf16": None, "e4m3": (4, 3), "e5m2": (5, 2), "e2m1": (2, 1)}
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def grid(store):
    return None if GRIDS[store] is None else F.grid_minifloat(*GRIDS[store])


def oracle_grid(store):
    e, m = GRIDS[store]
    return O.fp8(e, m) if e + m == 7 else O.minifloat(e, m)


def row_bytes(store, dim):
    return dim * {"bf16": 4, "e4m3": 2, "e5m2": 2, "e2m1": 1}[store] // 2


def new_cache(store, scales, pages, heads, size, dim, order="phs", fill=None):
    """A cache on the GPU whose dimensions (page, head, slot) lie in memory in `order`, filled with bytes of `fill`."""
    width = row_bytes(store, dim)
    count = {"p": pages, "h": heads, "s": size}

    def rows():
        t = torch.empty([count[c] for c in order] + [width], dtype=torch.uint8, device=DEV)
        t.fill_(0xAA if fill is None else fill)
        t = t.permute(*[order.index(c) for c in "phs"], 3)
        return t.view(torch.bfloat16) if store == "bf16" else t
    ks = vs = g = None
    if scales == "given":
        ks, vs = torch.full((1,), 0.031, device=DEV), torch.full((1,), 0.0123, device=DEV)
        g = F.gran("tensor")
    elif scales != "none":
        ks, vs = (torch.full((pages, heads, size), math.nan, dtype=torch.float16 if scales == "f16" else torch.float32, device=DEV) for _ in range(2))
        g = F.gran("row", scale_dtype=scales)
    return F.KVCache(rows(), rows(), ks, vs, grid(store), g)


def values(store, rows, scales):
    """Values (binary64) of rows of codes (numpy uint8 [..., bytes]) with a scale each."""
    if store == "bf16":
        return torch.from_numpy(np.ascontiguousarray(rows)).view(torch.bfloat16).double().numpy()
    codes = O.unpack_codes(rows.reshape(-1, rows.shape[-1]), oracle_grid(store))
    if store == "e2m1":
        table = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
        v = table[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    else:
        kind = torch.float8_e4m3fn if store == "e4m3" else torch.float8_e5m2
        v = torch.from_numpy(np.ascontiguousarray(codes.astype(np.uint8))).view(kind).double().numpy()
    s = np.asarray(scales, dtype=np.float64)
    return v.reshape(*rows.shape[:-1], -1) * (s if s.size == 1 else s[..., None])


def host(t):
    """Bytes or numbers of a tensor on the host."""
    t = t.detach().cpu()
    return t.contiguous().view(torch.uint8).numpy() if t.dtype in (torch.bfloat16, torch.uint8) else t.numpy()


def oracle_rows(store, scales, x, given):
    """What rows x (binary32 [n, dim]) become: bytes, scales."""
    if store == "bf16":
        return torch.from_numpy(x).bfloat16().view(torch.uint8).numpy(), None
    if scales == "given":
        codes, _ = O.quantize_pack(x, oracle_grid(store), "tensor", tensor_scale=given)
        return codes, None
    return O.quantize_pack(x, oracle_grid(store), "row", scale_dtype=scales)


# ---------------------------------------------------------------- rows in and out -----
ROWS = [("bf16", "none", 64, 16), ("bf16", "none", 192, 32), ("e4m3", "f32", 128, 16), ("e4m3", "f16", 96, 64), ("e4m3", "given", 256, 16),
        ("e5m2", "f32", 192, 32), ("e5m2", "f16", 64, 16), ("e5m2", "given", 128, 128), ("e2m1", "f32", 128, 16), ("e2m1", "f16", 96, 16),
        ("e2m1", "given", 64, 32), ("e2m1", "f16", 256, 16), ("e4m3", "f32", 192, 16), ("e2m1", "f32", 192, 256)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("store,scales,dim,size", ROWS)
def test_write_and_read(store, scales, dim, size, dtype):
    """Columns of wider rows go in, into pages in no order, of a cache laid out as [page, slot, head]; padding,
    positions past the table, absent pages and sequences have no row.  Codes and scales are the oracle's bit for bit, all
    other bytes stay, and reading gives the values, rounded once."""
    say("write and read", store, scales, dim, size, dtype)
    g = gen(1)
    heads, pages, max_pages, sequences, tokens = 3, 9, 3, 4, 61
    cache = new_cache(store, scales, pages, heads, size, dim, "psh")
    table = torch.tensor([[4, 0, -1], [7, 2, 8], [99, 1, -2 ** 31], [5, 3, 2 ** 31 - 1]], dtype=torch.int32)
    # distinct places, then some without a row
    places = torch.randperm(sequences * max_pages * size, generator=g)[:tokens - 6]
    seq = torch.cat([places // (max_pages * size), torch.tensor([0, 1, 4, -1, 2, 2 ** 31 - 1])]).to(torch.int32)
    pos = torch.cat([places % (max_pages * size), torch.tensor([-1, max_pages * size, 0, 3, -2 ** 31, 2 ** 31 - 1])]).to(torch.int32)
    rows = torch.randn(tokens, 3 * heads + 1, dim, generator=g) * torch.exp2(3 * torch.randn(tokens, 3 * heads + 1, 1, generator=g))
    rows[3, :, :] = 0.0
    rows[4, :, 1:] = 0.0
    rows[5] *= 1e-30
    rows = rows.to(DTYPES[dtype])
    wide = rows.to(DEV)
    k, v = wide[:, 1:1 + heads], wide[:, 1 + heads:1 + 2 * heads]
    before = [host(t).copy() for t in (cache.k, cache.v)]
    F.fp4_cache_write(k, v, cache, table.to(DEV), pos.to(DEV), seq.to(DEV))
    x = [rows[:, a:a + heads].float().numpy() for a in (1, 1 + heads)]
    given = [None if t is None else t.cpu().numpy() for t in (cache.k_scales, cache.v_scales)]
    want_rows, want_scales = [b.reshape(pages, heads, size, -1) for b in before], [np.full((pages, heads, size), np.nan) for _ in range(2)]
    live = []
    for i in range(tokens):
        s, p = int(seq[i]), int(pos[i])
        page = int(table[s, p // size]) if 0 <= s < sequences and 0 <= p < max_pages * size else -1
        live.append((page, p % size) if 0 <= page < pages else None)
    for j in range(2):
        codes, s = oracle_rows(store, scales, np.ascontiguousarray(x[j].reshape(-1, dim)), None if given[j] is None else given[j].ravel()[0])
        codes = codes.reshape(tokens, heads, -1)
        for i, at in enumerate(live):
            if at:
                want_rows[j][at[0], :, at[1]] = codes[i]
                if s is not None:
                    want_scales[j][at[0], :, at[1]] = s.reshape(tokens, heads)[i]
    for j, (t, s) in enumerate(((cache.k, cache.k_scales), (cache.v, cache.v_scales))):
        assert np.array_equal(host(t).reshape(pages, heads, size, -1), want_rows[j])
        if scales in ("f32", "f16"):
            assert np.array_equal(s.double().cpu().numpy(), want_scales[j], equal_nan=True)
    for out in ("f32", "bf16"):
        got = F.fp4_cache_read(cache, table.to(DEV), pos.to(DEV), seq.to(DEV), dtype=DTYPES[out])
        for j in range(2):
            want = np.zeros((tokens, heads, dim))
            for i, at in enumerate(live):
                if at:
                    s = 1.0 if store == "bf16" else given[j] if scales == "given" else want_scales[j][at[0], :, at[1]]
                    want[i] = values(store, want_rows[j][at[0], :, at[1]], s)
            # the product of a code's and a scale's significands rounds once to binary32
            want = torch.from_numpy(want).float().to(DTYPES[out])
            assert torch.equal(got[j].cpu(), want)


def test_write_is_the_quantizers():
    """Codes and scales as fp4_quantize_pack's, over half a million rows."""
    say("write against the quantizer")
    for store, scales in (("e4m3", "f32"), ("e2m1", "f16"), ("e5m2", "f16"), ("e2m1", "f32")):
        tokens, heads, dim, size = 65536, 4, 128, 64
        g = torch.Generator(device=DEV)
        g.manual_seed(3)
        x = torch.randn(2, tokens, heads, dim, device=DEV, generator=g) * torch.exp2(2 * torch.randn(2, tokens, heads, 1, device=DEV, generator=g))
        cache = F.kv_cache(tokens // size, heads, size, dim, grid(store), F.gran("row", scale_dtype=scales))
        table = torch.arange(tokens // size, dtype=torch.int32, device=DEV)[None]
        pos = torch.arange(tokens, dtype=torch.int32, device=DEV)
        F.fp4_cache_write(x[0], x[1], cache, table, pos, torch.zeros_like(pos))
        for t, (rows, s) in zip(x, ((cache.k, cache.k_scales), (cache.v, cache.v_scales))):
            p, q = F.fp4_quantize_pack(t.view(-1, dim), grid(store), F.gran("row", scale_dtype=scales))
            assert torch.equal(rows.transpose(1, 2).reshape(tokens * heads, -1), p)
            assert torch.equal(s.transpose(1, 2).reshape(-1), q.view(-1))


@pytest.mark.parametrize("store,scales", [("e4m3", "f32"), ("e4m3", "f16"), ("e5m2", "f32"), ("e2m1", "f16"), ("e2m1", "f32")])
def test_write_at_the_ends_of_scales(store, scales):
    """Rows of the smallest and largest magnitudes: scales stay finite, values read back finite, zeros stay zeros."""
    say("write tiny and huge", store, scales)
    top = {"e4m3": 448.0, "e5m2": 57344.0, "e2m1": 6.0}[store]
    peaks = [0.0, 1e-45, 1e-40, 2.0 ** -127, 2.0 ** -126 * top, 1e-30, 65504.0 * top * 0.99, 65504.0 * top * 1.5, 3.0e38]
    x = torch.zeros(len(peaks), 1, 64, device=DEV)
    x[:, 0, 3] = torch.tensor(peaks, device=DEV)
    x[:, 0, 7] = -torch.tensor(peaks, device=DEV) / 2
    cache = F.kv_cache(1, 1, 16, 64, grid(store), F.gran("row", scale_dtype=scales))
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    pos = torch.arange(len(peaks), dtype=torch.int32, device=DEV)
    F.fp4_cache_write(x, x, cache, table, pos, torch.zeros_like(pos))
    k, v = F.fp4_cache_read(cache, table, pos, torch.zeros_like(pos), dtype=torch.float32)
    assert torch.equal(k, v) and bool(torch.isfinite(k).all()) and bool(torch.isfinite(cache.k_scales.float()).all())
    assert bool((k[:, :, 8:] == 0).all()) and bool((k[0] == 0).all())
    for i, peak in enumerate(peaks):
        s = cache.k_scales[0, 0, i].double().item()
        assert (s == 0) == (peak == 0 or (scales == "f16" and peak / top <= 2.0 ** -25)), (peak, s)
        if scales == "f32" and peak >= 2.0 ** -126 * top or scales == "f16" and 1e-4 < peak / top < 65504:
            assert k[i, 0, 3].item() == pytest.approx(peak, rel=2.0 ** -10)


# ---------------------------------------------------------------- attention -----------
def sequence_rows(store, scales, cache, pages, lo, hi):
    """Keys and values (binary64 [heads, positions, dim]) and whether each position is there."""
    size = cache.page_size
    there = [0 <= int(pages[t // size]) < cache.k.shape[0] for t in range(lo, hi)]
    out = []
    for t, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        at = torch.tensor([int(pages[p // size]) if ok else 0 for p, ok in zip(range(lo, hi), there)], dtype=torch.long)
        slot = torch.arange(lo, hi) % size
        rows = host(t[at.to(DEV), :, slot.to(DEV)]).reshape(hi - lo, cache.kv_heads, -1)
        sc = 1.0 if s is None else s.cpu().numpy() if s.numel() == 1 else s[at.to(DEV), :, slot.to(DEV)].cpu().numpy()
        out.append(torch.from_numpy(values(store, rows, sc)).transpose(0, 1))
    return out[0], out[1], torch.tensor(there, dtype=torch.bool)


def reference(q, store, scales, cache, table, lengths, scale, window, most):
    """y, lse, and the bound's pieces: sum of p |V|, and the largest sum of |q k| times the scale."""
    n, heads, dim = q.shape
    share = heads // cache.kv_heads
    y, a = torch.zeros(n, heads, dim, dtype=torch.float64), torch.zeros(n, heads, dim, dtype=torch.float64)
    lse, reach = torch.full((n, heads), -math.inf, dtype=torch.float64), torch.zeros(n, heads, dtype=torch.float64)
    qd = q.detach().cpu().double().view(n, cache.kv_heads, share, dim)
    table = table.cpu()
    for b in range(n):
        hi = max(0, min(int(lengths[b]), most, table.shape[1] * cache.page_size))
        lo = max(0, hi - window) if window else 0
        if hi == lo:
            continue
        k, v, there = sequence_rows(store, scales, cache, table[b], lo, hi)
        if not there.any():
            continue
        k, v = k[:, there], v[:, there]
        for h in range(cache.kv_heads):
            z = (qd[b, h] @ k[h].T) * scale
            p = torch.softmax(z, 1)
            at = slice(h * share, (h + 1) * share)
            y[b, at], a[b, at], lse[b, at] = p @ v[h], p @ v[h].abs(), torch.logsumexp(z, 1)
            reach[b, at] = (qd[b, h].abs() @ k[h].abs().T).amax(1) * abs(scale)
    return y, lse, a, reach


def check(y, lse, ref, dim, length, wide, dtype):
    """Every z is off by at most dz: `dim` products exact in binary32 are added in `dim` steps, each within a whole step (2 U) of
    the largest partial sum, at most `reach`; the factors (scale, log2 e, the row's scale) round 4 times, and the exponential
    is within 2 U relative and reads a rounded difference (U |z - m|, at most 2 U reach).  The weights are
    off by dz + 3 U relative, their bf16 terms by 2^-18 (two) or 2^-27 (three); sums over the positions add at most `length` + 64
    roundings, to numerator (2 U, the matrix cores') and denominator (U) each; the quotient and the joins' factors 16 U.  All relative to
    sum p |V|, as the numerator's terms are.  The output rounds by half a step."""
    want, want_lse, a, reach = ref
    dz = ((2 * dim + 12) * U * reach)[..., None]
    rel = 2 * dz + (2.0 ** -27 if wide else 2.0 ** -18) + (3 * (length + 64) + 32) * U
    tol = rel * a + torch.finfo(dtype).eps / 2 * (want.abs() + rel * a) + 1e-37
    got = y.detach().cpu().double()
    off = (got - want).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((off <= tol).all()), (off - tol).max().item()
    if lse is not None:
        got = lse.cpu().double()
        empty = want_lse == -math.inf
        assert torch.equal(got == -math.inf, empty)
        # log of a sum within rel, plus dz itself and roundings of m, log and their sum
        tol = dz[..., 0] * 2 + ((length + 64) + 16) * U + 8 * U * want_lse.abs().nan_to_num(0, 0, 0) + 4 * U * reach
        assert bool(((got - want_lse).abs()[~empty] <= tol[~empty]).all())


def filled(store, scales, pages, heads, size, dim, seed, order="phs", std=1.0):
    """A cache all of whose rows were written (through the library: test_write_and_read holds it to the oracle)."""
    cache = new_cache(store, scales, pages, heads, size, dim, order)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = std * torch.randn(2, pages * size, heads, dim, device=DEV, generator=g)
    pos = torch.arange(pages * size, dtype=torch.int32, device=DEV)
    F.fp4_cache_write(x[0], x[1], cache, torch.arange(pages, dtype=torch.int32, device=DEV)[None], pos, torch.zeros_like(pos))
    return cache


def tables(lengths, size, pages, seed, spare=1):
    """A table whose used entries are distinct pages, the others -1."""
    order = torch.randperm(pages, generator=gen(seed)).to(torch.int32)
    most = max(-(-n // size) for n in lengths) + spare
    table, at = torch.full((len(lengths), most), -1, dtype=torch.int32), 0
    for i, n in enumerate(lengths):
        c = -(-max(n, 0) // size)
        table[i, :c] = order[at:at + c]
        at += c
    assert at <= pages
    return table.to(DEV)


SHORT = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("store,scales", [("bf16", "none"), ("e4m3", "f32"), ("e4m3", "f16"), ("e5m2", "given"), ("e5m2", "f32"), ("e2m1", "f16"),
                                          ("e2m1", "given")])
@pytest.mark.parametrize("dim,heads,share,size", [(64, 3, 1, 16), (96, 2, 5, 32), (128, 2, 8, 16), (128, 1, 20, 64), (192, 2, 16, 16), (256, 1, 7, 128)])
def test_attend_short(store, scales, dim, heads, share, size, dtype):
    """Lengths around every tile, half and workgroup border, all in one call, one sequence empty."""
    say("attend short", store, scales, dim, heads, share, size, dtype)
    pages = sum(-(-n // size) for n in SHORT) + 2
    cache = filled(store, scales, pages, heads, size, dim, 5)
    table = tables(SHORT, size, pages, 6)
    q = (2 * torch.randn(len(SHORT), heads * share, dim, generator=gen(7))).to(DTYPES[dtype]).to(DEV)
    lengths = torch.tensor(SHORT, dtype=torch.int32, device=DEV)
    lse = torch.full((len(SHORT), heads * share), math.nan, device=DEV)
    y = F.fp4_attend(q, cache, table, lengths, lse=lse)
    ref = reference(q, store, scales, cache, table, SHORT, dim ** -0.5, 0, 1 << 30)
    check(y, lse, ref, dim, max(SHORT), dtype == "f32", y.dtype)
    assert bool((y[0] == 0).all()) and torch.equal(y, F.fp4_attend(q, cache, table, lengths))


@pytest.mark.parametrize("store,scales,dim,size", [("e4m3", "f32", 128, 16), ("bf16", "none", 64, 64), ("e2m1", "f16", 128, 256), ("e5m2", "given", 96, 32),
                                                   ("bf16", "none", 256, 16), ("e2m1", "f32", 192, 16), ("e4m3", "f16", 256, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [0, 700])
def test_attend_long(store, scales, dim, size, dtype, window):
    """Sequences of several parts beside short ones: the parts are joined."""
    say("attend long", store, scales, dim, size, dtype, window)
    lengths = [5003, 512, 1, 513, 4096, 0, 1500, 2047]
    heads, share = 2, 3
    pages = sum(-(-n // size) for n in lengths) + 2
    cache = filled(store, scales, pages, heads, size, dim, 11)
    table = tables(lengths, size, pages, 12)
    q = (2 * torch.randn(len(lengths), heads * share, dim, generator=gen(13))).to(DTYPES[dtype]).to(DEV)
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    lse = torch.empty(len(lengths), heads * share, device=DEV)
    y = F.fp4_attend(q, cache, table, n, window=window, max_length=5003, lse=lse)
    ref = reference(q, store, scales, cache, table, lengths, dim ** -0.5, window, 5003)
    check(y, lse, ref, dim, 5003, dtype == "f32", y.dtype)
    again = F.fp4_attend(q, cache, table, n, window=window, max_length=5003)
    assert torch.equal(y, again)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 199, 200, 201, 10 ** 6, 2 ** 40])
def test_attend_windows(window):
    say("attend window", window)
    cache = filled("e4m3", "f32", 100, 2, 16, 64, 21)
    table = tables(SHORT, 16, 100, 22)
    q = torch.randn(len(SHORT), 6, 64, generator=gen(23)).to(DEV)
    lse = torch.empty(len(SHORT), 6, device=DEV)
    y = F.fp4_attend(q, cache, table, torch.tensor(SHORT, dtype=torch.int32, device=DEV), window=window, scale=0.3, lse=lse)
    check(y, lse, reference(q, "e4m3", "f32", cache, table, SHORT, 0.3, window, 1 << 30), 64, 200, True, y.dtype)


@pytest.mark.parametrize("y_dtype,q_dtype", [("f32", "bf16"), ("bf16", "f32")])
def test_attend_types(y_dtype, q_dtype):
    """q and y of different types; y given, its rows apart and what lies between them left alone; q columns of wider rows."""
    say("attend types", y_dtype, q_dtype)
    lengths = [77, 300, 5]
    cache = filled("e4m3", "f32", 30, 4, 16, 128, 31)
    table = tables(lengths, 16, 30, 32)
    wide = torch.randn(3, 20, 128, generator=gen(33)).to(DTYPES[q_dtype]).to(DEV)
    q = wide[:, 4:12]
    room = torch.full((3, 11, 128), 7.0, dtype=DTYPES[y_dtype], device=DEV)
    y = F.fp4_attend(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device=DEV), y=room[:, 2:10])
    check(y, None, reference(q, "e4m3", "f32", cache, table, lengths, 128 ** -0.5, 0, 1 << 30), 128, 300, True, y.dtype)
    assert bool((room[:, :2] == 7).all()) and bool((room[:, 10:] == 7).all())
    other = F.fp4_attend(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device=DEV), y_dtype=DTYPES[y_dtype])
    assert torch.equal(other, y)


@pytest.mark.parametrize("store,scales,fill", [("bf16", "none", 0xFF), ("e4m3", "f32", 0x7F), ("e5m2", "f16", 0x7C), ("e2m1", "f16", 0xFF)])
@pytest.mark.parametrize("order", ["phs", "psh", "hps", "shp"])
def test_attend_over_anything(store, scales, fill, order):
    """Rows that no sequence sees hold NaN or infinite codes and NaN scales, in any memory order; entries of the table past a sequence's end
    name pages that are not there; pages inside a sequence that are not in the cache are not seen; lengths are negative or
    past the table."""
    say("attend over anything", store, scales, order)
    size, dim, heads, pages = 16, 64, 2, 40
    cache = new_cache(store, scales, pages, heads, size, dim, order, fill)
    lengths = [40, 1, 100, 7, -5, 2 ** 31 - 1, 90, 0]
    table = torch.full((len(lengths), 7), 2 ** 31 - 1, dtype=torch.int32)
    table[0, :3] = torch.tensor([3, 39, 5])
    table[1, :1] = 0
    table[2, :7] = torch.tensor([8, -1, 9, 10, 40, 11, 12])  # two that are not there
    table[3, :1] = 13
    table[5, :7] = torch.arange(14, 21)
    table[6, :6] = torch.tensor([-2 ** 31, 100, -7, 2 ** 30, 41, -1])  # none there: nothing is seen
    g = gen(41)
    tokens = [(b, t) for b, n in enumerate(lengths) for t in range(max(0, min(n, 7 * size)))]
    seq, pos = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in zip(*tokens))
    x = torch.randn(2, len(tokens), heads, dim, generator=g).to(DEV)
    table = table.to(DEV)
    F.fp4_cache_write(x[0], x[1], cache, table, pos, seq)
    for dtype in ("bf16", "f32"):
        q = (3 * torch.randn(len(lengths), heads * 3, dim, generator=g)).to(DTYPES[dtype]).to(DEV)
        for window in (0, 50, 3):
            lse = torch.empty(len(lengths), heads * 3, device=DEV)
            y = F.fp4_attend(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device=DEV), window=window, lse=lse)
            ref = reference(q, store, scales, cache, table, lengths, dim ** -0.5, window, 1 << 30)
            check(y, lse, ref, dim, 112, dtype == "f32", y.dtype)
            for b in (4, 6, 7):
                assert bool((y[b] == 0).all()) and bool((lse[b] == -math.inf).all())


def test_attend_extreme_scores():
    """Scores of thousands, rising and falling along the sequence: the maximum moves at every tile, or never."""
    say("attend extreme scores")
    dim, size, n = 64, 16, 1500
    for sign in (1.0, -1.0):
        cache = new_cache("bf16", "none", 100, 1, size, dim)
        k = torch.zeros(n, 1, dim)
        k[:, 0, 0] = sign * torch.linspace(-40, 40, n)
        k = k.bfloat16()
        v = torch.randn(n, 1, dim, generator=gen(51)).bfloat16()
        table = torch.arange(100, dtype=torch.int32, device=DEV)[None]
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        F.fp4_cache_write(k.to(DEV), v.to(DEV), cache, table, pos, torch.zeros_like(pos))
        q = torch.zeros(1, 4, dim)
        q[0, :, 0] = torch.tensor([100.0, -100.0, 1.0, 0.01])
        q = q.to(DEV)
        lse = torch.empty(1, 4, device=DEV)
        y = F.fp4_attend(q, cache, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale=1.0, lse=lse)
        check(y, lse, reference(q, "bf16", "none", cache, table, [n], 1.0, 0, n), dim, n, True, y.dtype)


def test_attend_far_apart():
    """A cache of over 4 GiB, its pages and its heads more than 2^32 bytes apart."""
    say("attend far apart")
    lengths, dim, size = [50, 20], 128, 16
    for stride_page, stride_head, extent in ((size * dim * 4, 3 << 30, 7 << 30), (3 << 30, size * dim * 2, 7 << 30)):
        pages = 7 if stride_head > stride_page else 3
        raw = torch.empty(extent // 2, dtype=torch.bfloat16, device=DEV)
        other = torch.empty_like(raw)
        stride = (stride_page // 2, stride_head // 2, dim, 1)
        cache = F.KVCache(raw.as_strided((pages, 2, size, dim), stride), other.as_strided((pages, 2, size, dim), stride))
        table = torch.tensor([[6, 0, 3, 2], [1, 5, -1, -1]] if pages == 7 else [[2, 0, -1, -1], [1, -1, -1, -1]], dtype=torch.int32, device=DEV)
        g = gen(61)
        tokens = [(b, t) for b, n in enumerate(lengths) for t in range(n)]
        seq, pos = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in zip(*tokens))
        x = torch.randn(2, len(tokens), 2, dim, generator=g).bfloat16().to(DEV)
        F.fp4_cache_write(x[0], x[1], cache, table, pos, seq)
        k, v = F.fp4_cache_read(cache, table, pos, seq)
        live = (table[seq.long(), (pos // size).long()] >= 0)[:, None, None]
        assert torch.equal(k, torch.where(live, x[0], 0.0)) and torch.equal(v, torch.where(live, x[1], 0.0))
        q = torch.randn(2, 4, dim, generator=g).bfloat16().to(DEV)
        y = F.fp4_attend(q, cache, table, torch.tensor(lengths, dtype=torch.int32, device=DEV))
        check(y, None, reference(q, "bf16", "none", cache, table, lengths, dim ** -0.5, 0, 64), dim, 50, False, y.dtype)
        del raw, other, cache


def test_drafted_tokens():
    """Several new tokens of a sequence are sequences with its pages and a length each."""
    say("drafted tokens")
    cache = filled("e4m3", "f32", 40, 2, 16, 128, 71)
    table = tables([500], 16, 40, 72)
    lengths = [496, 497, 498, 499, 500]
    q = torch.randn(5, 8, 128, generator=gen(73)).bfloat16().to(DEV)
    shared = table.expand(5, -1)
    y = F.fp4_attend(q, cache, shared, torch.tensor(lengths, dtype=torch.int32, device=DEV))
    check(y, None, reference(q, "e4m3", "f32", cache, shared, lengths, 128 ** -0.5, 0, 1 << 30), 128, 500, False, y.dtype)
