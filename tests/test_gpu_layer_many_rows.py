"""Row, block and tile counts whose threads pass 2^32, the most that one launch takes: the call
splits them, and its results are those of smaller calls."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F = pytest.importorskip("bit_floating_point_amd")
DEV = "cuda"
E4 = (4, 3)


def say(*a):
    print(*a, flush=True)


def grid():
    return F.grid_minifloat(*E4)


def randn(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.empty(*shape, dtype=dtype, device=DEV).normal_(generator=g)


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("mode,group,scale_dtype", [("row", 0, "f32"), ("group", 8, "f16"), ("tensor", 0, "f32")])
def test_norm(mode, group, scale_dtype):
    """64 threads a row: 2^26 rows."""
    rows, cols, half = (1 << 26) + 5, 8, 1 << 25
    say("norm", rows, mode)
    x, gamma = randn(1, rows, cols), torch.ones(cols, device=DEV)
    residual = randn(2, rows, cols)
    ts = torch.full((1,), 0.01, device=DEV) if mode == "tensor" else None
    gr = F.gran(mode, group, scale_dtype)
    out, y = torch.empty_like(residual), torch.empty_like(x)
    p, s = F.fp4_rmsnorm_quant(x, gamma, grid(), gr, residual=residual, residual_out=out, y=y, tensor_scale=ts)
    for at in (slice(0, half), slice(half, rows)):
        o2, y2 = torch.empty_like(residual[at]), torch.empty_like(x[at])
        q, t = F.fp4_rmsnorm_quant(x[at], gamma, grid(), gr, residual=residual[at], residual_out=o2, y=y2, tensor_scale=ts)
        assert torch.equal(p[at], q) and torch.equal(out[at], o2) and torch.equal(y[at], y2)
        assert s is None or torch.equal(s[at], t)


def test_norm_of_terms():
    rows, cols, terms, half = (1 << 26) + 3, 8, 2, 1 << 25
    say("norm of terms", rows)
    x, gamma = randn(3, rows * terms, cols), torch.ones(cols, device=DEV)
    w = randn(4, rows, terms, dtype=torch.float32)
    y = torch.empty(rows, cols, device=DEV)
    F.fp4_rmsnorm_quant(x, gamma, terms=terms, term_weights=w, y=y)
    for a, b in ((0, half), (half, rows)):
        y2 = torch.empty(b - a, cols, device=DEV)
        F.fp4_rmsnorm_quant(x[a * terms:b * terms], gamma, terms=terms, term_weights=w[a:b], y=y2)
        assert torch.equal(y[a:b], y2)


@pytest.mark.parametrize("mode,group", [("row", 0), ("group", 512)])
def test_swiglu(mode, group):
    """64 threads a row for row scales, and for groups of 512 columns."""
    rows, cols, half = (1 << 26) + 5, 8, 1 << 25
    say("swiglu", rows, mode)
    x = randn(5, rows, 2 * cols)
    p, s = F.fp4_swiglu_quant(x, grid(), F.gran(mode, group))
    for at in (slice(0, half), slice(half, rows)):
        q, t = F.fp4_swiglu_quant(x[at], grid(), F.gran(mode, group))
        assert torch.equal(p[at], q) and torch.equal(s[at], t)


def test_quantize_block():
    """256 threads a block: 2^24 blocks, of many matrices and of one long one."""
    count, half = (1 << 24) + 5, 1 << 23
    say("quantize_block", count)
    w = randn(6, count, 1, 8)
    p, s = F.fp4_quantize_block(w, grid())
    for at in (slice(0, half), slice(half, count)):
        q, t = F.fp4_quantize_block(w[at], grid())
        assert torch.equal(p[at], q) and torch.equal(s[at], t)
    del w, p, s, q, t
    n, half = 128 * count - 100, 128 << 23
    w = randn(7, n, 8)
    p, s = F.fp4_quantize_block(w, grid())
    for a, b in ((0, half), (half, n)):
        q, t = F.fp4_quantize_block(w[a:b], grid())
        assert torch.equal(p[a:b], q) and torch.equal(s[a // 128:-(-b // 128)], t)


@pytest.mark.parametrize("M,N", [((1 << 30) + 70, 1), (1, (1 << 30) + 70), (3, (1 << 30) + 200)])
def test_product(M, N):
    """Tiles (streaming workgroups) of 256 threads: 2^24 of them.  The rows at both ends and around
    the middle, where a launch ends, are those of a small call."""
    K = 16
    say("product", M, N)
    a, w = torch.zeros(M, K, dtype=torch.uint8, device=DEV), torch.zeros(N, K, dtype=torch.uint8, device=DEV)
    sa, sw = torch.ones(M, 1, device=DEV), torch.ones(-(-N // 128), 1, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(8)
    long, scales = (a, sa) if M > N else (w, sw)
    count = max(M, N)
    spots = [0, 1 << 29, (1 << 30) - 512, (1 << 30) - 128, count - 40]
    for i, at in enumerate(spots):
        n = min(40, count - at)
        long[at:at + n] = (torch.randn(n, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
        if M > N:
            scales[at:at + n] = 2.0 ** (i - 2)
        else:
            scales[at // 128:(at + n - 1) // 128 + 1] = 2.0 ** (i - 2)
    short = w if M > N else a
    short[:] = (torch.randn(*short.shape, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
    y = F.fp4_gemm_block(a, sa, w, sw, grid(), grid())
    for at in spots:
        n = min(40, count - at)
        v = long[at:at + n].view(torch.float8_e4m3fn).double()
        v = v * (scales[at:at + n].double() if M > N else scales[torch.arange(at, at + n, device=DEV) // 128].double())
        ref = v @ short.view(torch.float8_e4m3fn).double().t()
        mag = v.abs() @ short.view(torch.float8_e4m3fn).double().abs().t()
        got = (y[at:at + n] if M > N else y[:, at:at + n].t()).double()
        # two sums of 16 products (window 7 * 2^-13 of the largest) and the rounding to bf16
        assert ((got - ref).abs() <= 2.0 ** -8 * ref.abs() + (7 * 2.0 ** -13 + 40 * 2.0 ** -24) * 1.01 * mag).all(), at
    middle = y[(1 << 29) + 64:(1 << 29) + 4096] if M > N else y[:, (1 << 29) + 64:(1 << 29) + 4096]
    assert not middle.any()


def test_experts():
    """The experts' columns, likewise: three slots of one expert."""
    N, K = (1 << 30) + 200, 16
    say("experts", N)
    w = torch.zeros(1, N, K, dtype=torch.uint8, device=DEV)
    sw = torch.ones(1, -(-N // 128), 1, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(9)
    a = (torch.randn(3, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
    offsets = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device=DEV)
    spots = [0, 1 << 29, (1 << 30) - 128, N - 40]
    for i, at in enumerate(spots):
        w[0, at:at + 40] = (torch.randn(40, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
        sw[0, at // 128:(at + 39) // 128 + 1] = 2.0 ** (i - 2)
    y = F.fp4_gemm_experts(a, torch.ones(3, 1, device=DEV), w, sw, grid(), grid(), offsets, slots)
    for at in spots:
        v = w[0, at:at + 40].view(torch.float8_e4m3fn).double() * sw[0, torch.arange(at, at + 40, device=DEV) // 128].double()
        av = a.view(torch.float8_e4m3fn).double()
        ref, mag = av @ v.t(), av.abs() @ v.abs().t()
        assert ((y[:, at:at + 40].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (7 * 2.0 ** -13 + 40 * 2.0 ** -24) * 1.01 * mag).all(), at
    assert not y[:, (1 << 29) + 64:(1 << 29) + 4096].any()
