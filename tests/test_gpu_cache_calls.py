"""How calls on a key/value cache can be made: captured and replayed while positions and lengths change, on other
streams and threads, with workspaces that are kept and shared, beside padding, at the ends of sizes and of
scales.  Oracle and bounds are those of test_gpu_cache.py."""
import math
import threading

import pytest
import torch

import bit_floating_point_amd as F
from bit_floating_point_amd.cache import _workspace_size
from test_gpu_cache import DEV, DTYPES, check, filled, gen, grid, new_cache, reference, say, tables

pytestmark = pytest.mark.gpu
I32 = torch.int32


def ints(values):
    return torch.tensor(values, dtype=I32, device=DEV)


# ---------------------------------------------------------------- graphs, streams, threads -----
@pytest.mark.parametrize("store,scales", [("bf16", "none"), ("e4m3", "f32"), ("e2m1", "f16")])
def test_replays_while_sequences_grow(store, scales):
    """A captured write and attention: positions, lengths, pages and rows change between the replays, some sequences of one part
    become sequences of several, and tokens turn into padding."""
    say("replays", store, scales)
    n, heads, share, dim, size, most = 4, 2, 3, 128, 16, 2048
    pages = n * most // size
    two = [filled(store, scales, pages, heads, size, dim, 5) for _ in range(2)]
    table = torch.randperm(pages, generator=gen(6)).to(I32).view(n, -1).to(DEV)
    x = torch.randn(2, n, heads, dim, generator=gen(7)).bfloat16().to(DEV)
    q = torch.randn(n, heads * share, dim, generator=gen(8)).bfloat16().to(DEV)
    positions, lengths, lse = ints([0] * n), ints([0] * n), torch.empty(n, heads * share, device=DEV)

    def calls(cache):
        F.fp4_cache_write(x[0], x[1], cache, table, positions)
        return F.fp4_attend(q, cache, table, lengths, lse=lse), F.fp4_cache_read(cache, table, positions)
    calls(two[0]), calls(two[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, (k, v) = calls(two[0])
    steps = [[0, 1, 2, 3], [15, 511, 512, 1023], [16, 1024, -1, 2047], [2047, 2047, 2047, 2047], [-1, 5, -1, 2048], [700, 1500, 40, 0]]
    for turn, at in enumerate(steps):
        g = gen(100 + turn)
        positions.copy_(ints(at))
        lengths.copy_(ints([p + 1 for p in at]))
        x.copy_(torch.randn(2, n, heads, dim, generator=g).bfloat16())
        q.copy_(torch.randn(n, heads * share, dim, generator=g).bfloat16())
        table.copy_(table.roll(turn, 0))
        if turn % 2:
            torch.cuda.synchronize()
        graph.replay()
        got = [t.clone() for t in (y, k, v, lse)]
        want, (wk, wv) = calls(two[1])
        assert all(torch.equal(a, b) for a, b in zip(got, (want, wk, wv, lse)))
        ref = reference(q, store, scales, two[1], table, [p + 1 for p in at], dim ** -0.5, 0, most)
        check(y, lse, ref, dim, most, False, y.dtype)
    assert torch.equal(two[0].k, two[1].k) and torch.equal(two[0].v, two[1].v)


def test_graphs_that_share_a_workspace():
    """Two captured calls of different sizes, one workspace, replayed in turn on one stream with eager calls that use it too."""
    say("shared workspace")
    size, dim = 16, 128
    cache = filled("e4m3", "f32", 600, 2, size, dim, 11)
    made = []
    need = 0
    for lengths, heads in (([4000, 700], 8), ([1, 2500, 0, 1100, 513], 4)):
        table = tables(lengths, size, 600, 12)
        q = torch.randn(len(lengths), heads, dim, generator=gen(13)).bfloat16().to(DEV)
        made.append((q, cache, table, ints(lengths)))
        need = max(need, _workspace_size(len(lengths), heads, 2, dim, table.shape[1] * size, 0))
    assert need > 0
    room = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    want = [F.fp4_attend(*a) for a in made]
    for a in made:
        F.fp4_attend(*a, workspace=room)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in made:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(F.fp4_attend(*a, workspace=room))
    for turn in range(6):
        for i in (turn % 2, 1 - turn % 2, turn % 2):
            outs[i].fill_(7)
            graphs[i].replay()
            assert torch.equal(outs[i], want[i])
        assert torch.equal(F.fp4_attend(*made[turn % 2], workspace=room), want[turn % 2])
        room.fill_(0x7F if turn % 2 else 0xFF)


def test_other_streams():
    """Calls go to the stream that is current, behind what it already has to do."""
    say("other streams")
    cache = filled("e4m3", "f32", 300, 2, 16, 128, 21)
    lengths = [2000, 1500, 40]
    table = tables(lengths, 16, 300, 22)
    q = torch.randn(3, 8, 128, generator=gen(23)).bfloat16().to(DEV)
    x = torch.randn(2, 3, 2, 128, generator=gen(24)).to(DEV)
    last, n = ints([v - 1 for v in lengths]), ints(lengths)
    F.fp4_cache_write(x[0], x[1], cache, table, last)
    want, (wk, wv) = F.fp4_attend(q, cache, table, n), F.fp4_cache_read(cache, table, last)
    other = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device=DEV)
    late_x, late_q = torch.zeros_like(x), torch.zeros_like(q)
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(3):
            a = a @ a * 1e-4  # keeps the stream busy while the calls below are made
        late_x.copy_(x + 0 * a.flatten()[:x.numel()].view_as(x))
        late_q.copy_(q)
        F.fp4_cache_write(late_x[1], late_x[0], cache, table, last)  # something else first
        F.fp4_cache_write(late_x[0], late_x[1], cache, table, last)
        y = F.fp4_attend(late_q, cache, table, n)
        k, v = F.fp4_cache_read(cache, table, last)
    other.synchronize()
    assert torch.equal(y, want) and torch.equal(k, wk) and torch.equal(v, wv)


def test_two_threads():
    """One cache, two threads with a stream each, at the same time."""
    say("two threads")
    cache = filled("e2m1", "f16", 300, 2, 16, 64, 31)
    work = []
    for i, lengths in enumerate(([2000, 30, 900], [1, 1700])):
        table = tables(lengths, 16, 300, 32 + i)
        q = torch.randn(len(lengths), 6, 64, generator=gen(34 + i)).to(DEV)
        work.append((q, cache, table, ints(lengths)))
    want = [F.fp4_attend(*a) for a in work]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(30):
                y = F.fp4_attend(*work[i])
                s.synchronize()
                if not torch.equal(y, want[i]):
                    wrong.append(i)
    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_the_same_bits_every_time():
    """Parts are joined in order, whatever finishes first; sequences in a batch do not change each other."""
    say("the same bits")
    lengths = [3000, 1, 2999, 700, 5000, 512, 4096, 33]
    cache = filled("e4m3", "f32", 1100, 2, 16, 128, 41)
    table = tables(lengths, 16, 1100, 42)
    q = torch.randn(len(lengths), 10, 128, generator=gen(43)).bfloat16().to(DEV)
    y = F.fp4_attend(q, cache, table, ints(lengths))
    for _ in range(20):
        assert torch.equal(y, F.fp4_attend(q, cache, table, ints(lengths)))
    order = torch.tensor([5, 0, 7, 2, 1, 4, 3, 6])
    again = F.fp4_attend(q[order.to(DEV)], cache, table[order.to(DEV)], ints([lengths[i] for i in order]))
    assert torch.equal(again, y[order.to(DEV)])


# ---------------------------------------------------------------- sizes -------------------------
@pytest.mark.parametrize("share", [15, 16, 17, 33, 64])
@pytest.mark.parametrize("store,scales,dtype", [("e4m3", "f32", "bf16"), ("bf16", "none", "f32"), ("e2m1", "f16", "bf16")])
def test_many_query_heads(share, store, scales, dtype):
    say("many query heads", share, store, dtype)
    lengths = [1300, 17, 600]
    cache = filled(store, scales, 160, 1, 16, 64, 51)
    table = tables(lengths, 16, 160, 52)
    q = (2 * torch.randn(3, share, 64, generator=gen(53))).to(DTYPES[dtype]).to(DEV)
    lse = torch.empty(3, share, device=DEV)
    y = F.fp4_attend(q, cache, table, ints(lengths), lse=lse)
    check(y, lse, reference(q, store, scales, cache, table, lengths, 0.125, 0, 1 << 30), 64, 1300, dtype == "f32", y.dtype)


@pytest.mark.parametrize("store,scales,size,length", [("e2m1", "f16", 65536, 70000), ("e5m2", "f32", 4096, 4097), ("bf16", "none", 1024, 1023)])
def test_large_pages(store, scales, size, length):
    say("large pages", store, size, length)
    cache = filled(store, scales, 2, 1, size, 64, 61)
    table = ints([[1, 0], [0, 1]])
    q = torch.randn(2, 2, 64, generator=gen(62)).bfloat16().to(DEV)
    for window in (0, 40):
        y = F.fp4_attend(q, cache, table, ints([length, 5]), window=window)
        check(y, None, reference(q, store, scales, cache, table, [length, 5], 0.125, window, 1 << 30), 64, length, False, y.dtype)


def test_more_sequences_than_a_grid_has():
    """70 000 sequences of up to 16 positions, and as many tokens written for them."""
    say("70000 sequences")
    n, pages, size, dim = 70000, 70000, 16, 64
    cache = new_cache("e4m3", "f32", pages, 1, size, dim)
    table = torch.randperm(pages, generator=gen(71)).to(I32)[:, None].to(DEV)
    lengths = (torch.arange(n) % 17).to(I32).to(DEV)
    x = torch.randn(2, n * size, 1, dim, device=DEV, generator=torch.Generator(device=DEV).manual_seed(72)).bfloat16()
    at = torch.arange(n * size, dtype=I32, device=DEV)
    live = at % size < lengths[at.long() // size]
    F.fp4_cache_write(x[0], x[1], cache, table, torch.where(live, at % size, -1).to(I32), at // size)
    k, v = F.fp4_cache_read(cache, table, at % size, at // size, dtype=torch.float32)
    k, v, live = k.view(n, size, dim), v.view(n, size, dim), live.view(n, size)
    q = torch.randn(n, 1, dim, generator=gen(73)).bfloat16().to(DEV)
    lse = torch.empty(n, 1, device=DEV)
    y = F.fp4_attend(q, cache, table, lengths, lse=lse)
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    kd, vd = (torch.where(live[..., None], t.double(), zero) for t in (k, v))
    z = torch.where(live, (kd * q.double()).sum(2) * 0.125, -math.inf)
    reach = ((kd * q.double()).abs().sum(2) * 0.125).amax(1, keepdim=True)
    want_lse = torch.logsumexp(z, 1, keepdim=True)
    p = torch.where(live, torch.exp(z - torch.where(want_lse == -math.inf, zero, want_lse)), zero)
    want, a = (p[..., None] * vd).sum(1, keepdim=True), (p[..., None] * vd.abs()).sum(1, keepdim=True)
    check(y, lse, [t.cpu() for t in (want, want_lse, a, reach)], dim, size, False, y.dtype)
    assert int((lse == -math.inf).sum()) == int((lengths == 0).sum()) and bool((y[lengths == 0] == 0).all())


def test_more_rows_than_a_launch_takes():
    """65 535 heads of 8196 tokens, a lane for each 8 values: over 2^32 threads.  Almost all tokens are padding; those around
    the border of the launches and at the ends are not.  Then the attention over so many heads."""
    say("8196 tokens of 65535 heads")
    tokens, heads, dim = 8196, 65535, 64
    cache = F.kv_cache(1, heads, 16, dim, grid("e2m1"), F.gran("row", scale_dtype="f16"))
    rows = torch.empty(tokens, heads, dim, dtype=torch.bfloat16, device=DEV)  # 69 GB, of which eight tokens mean something
    at = [0, 1, 8190, 8191, 8192, 8193, 8194, 8195]
    x = torch.randn(len(at), heads, dim, device=DEV, generator=torch.Generator(device=DEV).manual_seed(81)).bfloat16()
    rows[torch.tensor(at, device=DEV)] = x
    positions = torch.full((tokens,), -1, dtype=I32, device=DEV)
    positions[torch.tensor(at, device=DEV)] = torch.arange(len(at), dtype=I32, device=DEV)
    F.fp4_cache_write(rows, rows, cache, torch.zeros(1, 1, dtype=I32, device=DEV), positions, torch.zeros_like(positions))
    del rows
    codes, scales = F.fp4_quantize_pack(x.view(-1, dim), grid("e2m1"), F.gran("row", scale_dtype="f16"))
    for t, s in ((cache.k, cache.k_scales), (cache.v, cache.v_scales)):
        assert torch.equal(t[0, :, :len(at)].transpose(0, 1).reshape(-1, dim // 2), codes)
        assert torch.equal(s[0, :, :len(at)].t().reshape(-1), scales.view(-1))
        assert bool((t[0, :, len(at):] == 0).all())
    zeros = torch.zeros(1, 1, dtype=I32, device=DEV)
    k, v = F.fp4_cache_read(cache, zeros, ints(list(range(8))), ints([0] * 8), dtype=torch.float32)
    y = F.fp4_attend(x[:1].float(), cache, zeros, ints([8]), scale=0.125)
    kd, vd, qd = k.double(), v.double(), x[:1].double()
    p = torch.softmax((kd * qd).sum(2) * 0.125, 0)
    want, a = (p[..., None] * vd).sum(0, keepdim=True), (p[..., None] * vd.abs()).sum(0, keepdim=True)
    reach = ((kd * qd).abs().sum(2) * 0.125).amax(0, keepdim=True)
    check(y, None, [t.cpu() for t in (want, torch.zeros(1, heads, dtype=torch.float64), a, reach)], dim, 8, True, y.dtype)


def test_nothing_to_do():
    """No tokens, no sequences, no pages in the table: nothing is written; reads and results without rows are zeros."""
    say("nothing to do")
    cache = filled("e4m3", "f32", 4, 2, 16, 64, 91)
    before = cache.k.clone(), cache.v.clone(), cache.k_scales.clone()
    none, x = torch.zeros(0, 2, 64, device=DEV), torch.ones(3, 2, 64, device=DEV)
    F.fp4_cache_write(none, none, cache, torch.zeros(3, 1, dtype=I32, device=DEV), ints([]))
    F.fp4_cache_write(x, x, cache, torch.zeros(0, 1, dtype=I32, device=DEV), ints([0, 1, 2]))
    F.fp4_cache_write(x, x, cache, torch.zeros(3, 0, dtype=I32, device=DEV), ints([0, 1, 2]))
    assert torch.equal(cache.k, before[0]) and torch.equal(cache.v, before[1]) and torch.equal(cache.k_scales, before[2])
    k, v = F.fp4_cache_read(cache, torch.zeros(3, 0, dtype=I32, device=DEV), ints([0, 1, 2]))
    assert bool((k == 0).all()) and bool((v == 0).all())
    q, lse = torch.ones(3, 4, 64, device=DEV), torch.zeros(3, 4, device=DEV)
    for table, kw in ((torch.zeros(3, 0, dtype=I32, device=DEV), {}), (torch.zeros(3, 1, dtype=I32, device=DEV), dict(max_length=0))):
        y = F.fp4_attend(q, cache, table, ints([3, 1, 9]), lse=lse.fill_(3), **kw)
        assert bool((y == 0).all()) and bool((lse == -math.inf).all())
    assert F.fp4_attend(q[:0], cache, torch.zeros(0, 4, dtype=I32, device=DEV), ints([])).shape == (0, 4, 64)


# ---------------------------------------------------------------- scales ------------------------
@pytest.mark.parametrize("store,scales", [("e4m3", "f32"), ("e2m1", "f16"), ("bf16", "none"), ("e5m2", "given")])
def test_any_factor(store, scales):
    """Negative, zero, tiny and large factors of the products."""
    say("any factor", store)
    lengths = [600, 45, 1]
    cache = filled(store, scales, 60, 2, 16, 64, 95)
    table = tables(lengths, 16, 60, 96)
    q = torch.randn(3, 4, 64, generator=gen(97)).bfloat16().to(DEV)
    lse = torch.empty(3, 4, device=DEV)
    for scale in (-0.125, 0.0, 1e-30, 3.0, -40.0):
        y = F.fp4_attend(q, cache, table, ints(lengths), scale=scale, lse=lse)
        check(y, lse, reference(q, store, scales, cache, table, lengths, scale, 0, 1 << 30), 64, 600, False, y.dtype)


@pytest.mark.parametrize("store", ["e4m3", "e5m2", "e2m1"])
def test_given_scales(store):
    """A given scale of zero or less, and values beyond what it reaches: codes as the quantizer's."""
    say("given scales", store)
    x = torch.randn(2, 16, 1, 64, generator=gen(98)).to(DEV)
    at = torch.arange(16, dtype=I32, device=DEV)
    table, zeros = torch.zeros(1, 1, dtype=I32, device=DEV), torch.zeros(16, dtype=I32, device=DEV)
    for s in (0.0, -0.01, 1e-5, 0.5, 100.0):
        ks, vs = torch.full((1,), s, device=DEV), torch.full((1,), 2 * s, device=DEV)
        cache = F.kv_cache(1, 1, 16, 64, grid(store), k_scale=ks, v_scale=vs)
        F.fp4_cache_write(x[0], x[1], cache, table, at, zeros)
        for t, rows, scale in ((x[0], cache.k, ks), (x[1], cache.v, vs)):
            codes, _ = F.fp4_quantize_pack(t.view(16, 64), grid(store), F.gran("tensor"), tensor_scale=scale)
            assert torch.equal(rows[0, 0], codes), s


@pytest.mark.parametrize("store,scales", [("bf16", "none"), ("e4m3", "f32"), ("e5m2", "f32"), ("e2m1", "f16")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_values(store, scales, dtype):
    """Keys and values of very different sizes from row to row, scores kept small by q."""
    say("large and small values", store, dtype)
    n, top = 700, 10 if scales == "f16" else 60
    cache = new_cache(store, scales, 44, 1, 16, 64)
    g = gen(99)
    size = torch.exp2(torch.randint(-top, top + 1, (n, 1, 1), generator=g).float())
    k, v = (torch.randn(n, 1, 64, generator=g) * size[torch.randperm(n, generator=g)] for _ in range(2))
    table = torch.arange(44, dtype=I32, device=DEV)[None]
    at = torch.arange(n, dtype=I32, device=DEV)
    F.fp4_cache_write(k.to(DEV), v.to(DEV), cache, table, at, torch.zeros_like(at))
    q = (torch.randn(1, 3, 64, generator=g) * 2.0 ** -top).to(DTYPES[dtype]).to(DEV)
    lse = torch.empty(1, 3, device=DEV)
    y = F.fp4_attend(q, cache, table, ints([n]), lse=lse)
    check(y, lse, reference(q, store, scales, cache, table, [n], 0.125, 0, n), 64, n, dtype == "f32", y.dtype)
