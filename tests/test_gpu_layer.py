"""The layer operators (include/fp4_layer.h) against plain references in 64 bits.

u = 2^-24 is binary32's unit rounding.  Bounds, from the operations' own rounding counts:
  * the stream h = residual + sum_j w_j x_j, one fused multiply-add per term:
    |h32 - h| <= (terms + 1) u H, H = the same sum over magnitudes; stored bf16 adds 2^-8 |h|;
  * the normed row n = h r g, r = 1 / sqrt(mean(h^2) + eps): the sum of squares has at most
    64 + 6 + 16 additions on a path (a lane's 64 values, the lanes, the wavefronts), all
    terms positive, and r halves its relative error; with the squares, the division, the
    addition, the root, the reciprocal and two products r g adds at most
    (86 / 2 + 8) u = 51 u of |n|, and h's own error scales with r |g|, also through the
    sum of squares, where it is at most max_row(|h32 - h|) / rms(h) relative;
  * SwiGLU: e^-g is 2^t with t = g log2 e, whose rounding (constant and product, 2 u of |t|)
    gives 2 u |g| relative; the exponential and the reciprocal within 1 ulp (2 u) each, one
    addition and two products: (2 |g| + 8) u of |h|; gates below -87 give results under
    2^-100 |u|, where e^-g may overflow: an absolute 2^-100 |u|;
  * scales: the bound of the unit's largest value, the division, and binary16's 2^-11
    (2^-24 absolute) where they are stored so;
  * codes: x32 = n32 / s32 is within its bound e of n / s; the code must lie between the
    nearest codes of n/s - e and n/s + e (conversion is monotone);
  * products: the framework's bound of packed products, (2 K + 2 nb + 4) u S plus the
    matrix instruction's product window 7 * 2^-13 S (S = the product over magnitudes; one
    scale product and one fused multiply-add per block), and 1e-3 in norm;
  * routing weights: an exponential (argument within u |l|, so 2 u |l - top|; 2 ulp), sums of
    at most 22 + 6 additions, two divisions, one factor: (2 |l - top| + 40) u relative.
    Experts, offsets and slots are exact: inputs leave no choice to rounding.
"""
import math

import numpy as np
import pytest
import torch

import oracle as O

pytestmark = pytest.mark.gpu

F = pytest.importorskip("bit_floating_point_amd")
DEV = "cuda"
U = 2.0 ** -24
GRIDS = {"e4m3": (4, 3), "e5m2": (5, 2)}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
QMAX = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, flush=True)


def grid(name):
    return F.grid_minifloat(*GRIDS[name])


def rng(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F._lib.lib()
    yield
    torch.cuda.synchronize()


# ---------------------------------------------------------------- codes ----------------
def code_values(name):
    """All finite values of the grid, ascending, in 64 bits."""
    v = torch.arange(256, dtype=torch.uint8).view(FLOAT8[name]).double()
    v = v[torch.isfinite(v)]
    return torch.unique(v)


def nearest(name, x):
    """Largest and smallest nearest grid values of x (they differ on a tie)."""
    v = code_values(name)
    x = x.clamp(v[0], v[-1])
    hi = torch.searchsorted(v, x).clamp(1, len(v) - 1)
    lo = hi - 1
    down, up = x - v[lo], v[hi] - x
    return torch.where(down <= up, v[lo], v[hi]), torch.where(up <= down, v[hi], v[lo])


def check_codes(name, packed, scales, n, err, mode, group=0, f16=False, tensor_scale=None, shift=None):
    """Codes and scales of n (64 bits, each value known to within err)."""
    rows, cols = n.shape
    got = packed.cpu().view(FLOAT8[name]).double()
    assert torch.isfinite(got).all()
    if mode == "tensor":
        s = tensor_scale.cpu().double() * 2.0 ** shift.cpu().double() if shift is not None else tensor_scale.cpu().double()
        s = s.expand(rows, cols)
    else:
        width = cols if mode == "row" else group
        units = -(-cols // width)
        pad = (0, units * width - cols)
        m = torch.nn.functional.pad(n.abs(), pad).view(rows, units, width)
        e = torch.nn.functional.pad(err, pad).view(rows, units, width)
        want = m.amax(2) / QMAX[name]
        slack = e.amax(2) / QMAX[name] + want * (2 * U + (2.0 ** -11 if f16 else 0)) + (2.0 ** -24 if f16 else 0)
        s32 = scales.cpu().double().view(rows, units)
        worst = ((s32 - want).abs() / slack.clamp_min(1e-300)).max().item()
        say(f"  scales: {worst:.3f} of the bound")
        assert worst <= 1.0
        s = s32.repeat_interleave(width, 1)[:, :cols]
    zero = s == 0
    x = torch.where(zero, 0.0, n / s.clamp_min(1e-300))
    e = torch.where(zero, 0.0, err / s.clamp_min(1e-300)) + 4 * U * x.abs()
    low, high = nearest(name, x - e)[0], nearest(name, x + e)[1]
    assert ((got >= low) & (got <= high)).all(), "a code is not the nearest one"


# ---------------------------------------------------------------- norm ----------------
def norm_reference(x, gamma, eps, residual, terms, weights):
    rows = x.shape[0] // terms
    xd = x.double().view(rows, terms, -1)
    if weights is not None:
        w = weights.double()[:, :, None]
        xd = torch.where(w == 0, 0.0, w * xd)
    h, H = xd.sum(1), xd.abs().sum(1)
    if residual is not None:
        h, H = h + residual.double(), H + residual.double().abs()
    eh = (terms + 1) * U * H
    ms = (h * h).mean(1, keepdim=True) + eps
    r = 1 / ms.sqrt()
    n = h * r * gamma.double()
    # h's errors e: sqrt(mean((h + e)^2)) moves by at most rms(e)
    rel = (eh * eh).mean(1, keepdim=True).sqrt() * r
    en = (eh * r * gamma.double().abs() + n.abs() * rel) * 1.01 + 51 * U * n.abs()
    return h, eh, n, en


def check_stream(out, h, eh):
    e = eh + (2.0 ** -8 * h.abs() if out.dtype == torch.bfloat16 else 0)
    d = (out.cpu().double() - h).abs()
    assert (d <= e).all(), (d / e.clamp_min(1e-300)).max()


NORM = [
    # rows, cols, terms, x, residual, gamma, y, grid, mode, group, f16
    (1, 5120, 1, "bf16", "bf16", "bf16", None, "e4m3", "row", 0, False),
    (3, 8, 1, "f32", "f32", "f32", "f32", "e4m3", "group", 8, False),
    (5, 520, 1, "bf16", None, "f32", "bf16", "e5m2", "group", 128, False),
    (33, 2080, 2, "bf16", "f32", "bf16", "bf16", "e4m3", "group", 128, True),
    (17, 1096, 8, "bf16", "bf16", "bf16", "bf16", "e4m3", "group", 512, False),
    (9, 11016, 1, "f32", "bf16", "f32", None, "e5m2", "tensor", 0, False),
    (2, 16384, 3, "f32", "f32", "bf16", "f32", "e4m3", "row", 0, True),
    (2, 65536, 1, "bf16", "bf16", "bf16", None, "e4m3", "group", 64, False),
    (700, 4096, 1, "bf16", "bf16", "bf16", None, "e4m3", "row", 0, False),
    (1300, 5120, 4, "bf16", "bf16", "bf16", "bf16", "e4m3", "group", 128, False),
    (4100, 264, 1, "bf16", "f32", "f32", None, "e4m3", "group", 32, False),
    (64, 24576, 6, "bf16", "bf16", "bf16", None, "e4m3", "group", 256, False),
]


@pytest.mark.parametrize("rows,cols,terms,xt,rt,gt,yt,fmt,mode,group,f16", NORM)
def test_norm(rows, cols, terms, xt, rt, gt, yt, fmt, mode, group, f16):
    say("norm", rows, cols, terms, xt, rt, gt, yt, fmt, mode, group)
    g = rng(rows + cols)
    x = randn(g, rows * terms, cols).to(TYPES[xt])
    gamma = (1 + 0.2 * randn(g, cols)).to(TYPES[gt])
    residual = (2 * randn(g, rows, cols)).to(TYPES[rt]) if rt else None
    weights = None
    if terms > 1:
        weights = torch.rand(rows, terms, generator=g)
        weights[torch.rand(rows, terms, generator=g) < 0.2] = 0.0
        x.view(rows, terms, cols)[weights == 0] = float("nan")  # absent terms may hold anything
    if rows > 2:
        x.view(rows, terms, cols)[1] = 0  # a row of zeros, unless the residual fills it
        if residual is not None:
            residual[1] = 0
    scale = torch.tensor([4.0 / QMAX[fmt]]) if mode == "tensor" else None
    shift = -torch.randint(0, 5, (cols,), generator=g).to(torch.int8) if mode == "tensor" else None
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    out = torch.full((rows, cols), 7.0, dtype=TYPES[rt] if rt else torch.float32, device=DEV)
    y = torch.empty(rows, cols, dtype=TYPES[yt], device=DEV) if yt else None
    packed, scales = F.fp4_rmsnorm_quant(to(x), to(gamma), grid(fmt), F.gran(mode, group, "f16" if f16 else "f32"), eps=1e-5,
                                         residual=to(residual), residual_out=out, terms=terms, term_weights=to(weights),
                                         tensor_scale=to(scale), col_shift=to(shift), y=y)
    h, eh, n, en = norm_reference(x, gamma, 1e-5, residual, terms, weights)
    check_stream(out, h, eh)
    if y is not None:
        check_stream(y, n, en)
    check_codes(fmt, packed, scales, n, en, mode, group, f16, scale, shift)


def test_norm_in_place_strides_and_parts():
    """residual_out = residual, padded rows, y alone, stream alone, weights of 1."""
    g = rng(5)
    rows, cols = 37, 328
    big = randn(g, rows, cols + 24).bfloat16().to(DEV)
    x = big[:, 8:8 + cols]
    gamma = torch.ones(cols, device=DEV)
    residual = randn(g, rows, cols + 8).bfloat16().to(DEV)[:, :cols]
    h, eh, n, en = norm_reference(x.cpu(), gamma.cpu(), 1e-6, residual.cpu(), 1, None)
    r1, y1 = torch.empty_like(residual), torch.empty(rows, cols + 16, device=DEV)[:, :cols]
    packed = torch.full((rows, cols + 40), 99, dtype=torch.uint8, device=DEV)
    p1, s1 = F.fp4_rmsnorm_quant(x, gamma, grid("e4m3"), F.gran("group", 128), residual=residual, residual_out=r1, y=y1,
                                 packed=packed[:, :cols])
    assert (packed[:, cols:] == 99).all()
    check_stream(r1, h, eh)
    check_stream(y1, n, en)
    check_codes("e4m3", p1, s1, n, en, "group", 128)
    y2, r2 = torch.empty(rows, cols, device=DEV), residual.clone()
    F.fp4_rmsnorm_quant(x, gamma, residual=residual, y=y2)
    assert torch.equal(y2, y1)
    F.fp4_rmsnorm_quant(x, gamma, residual=r2, residual_out=r2)
    assert torch.equal(r2, r1)
    p3, s3 = F.fp4_rmsnorm_quant(x, gamma, grid("e4m3"), F.gran("group", 128), residual=residual, residual_out=residual,
                                 term_weights=torch.ones(rows, 1, device=DEV))
    assert torch.equal(residual, r1) and torch.equal(p3, p1.contiguous()) and torch.equal(s3, s1)


def test_norm_empty():
    for rows, cols in ((0, 256), (4, 0)):
        p, s = F.fp4_rmsnorm_quant(torch.empty(rows, cols, device=DEV), torch.empty(cols, device=DEV), grid("e4m3"), F.gran("row"))
        assert p.shape == (rows, cols)


def test_norm_past_32_bits():
    """A stream of more than 2^31 values: the last rows are those of a small call."""
    rows, cols = 280000, 8192
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    tail = randn(rng(1), 5, cols).bfloat16().to(DEV)
    x[-5:] = tail
    gamma = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    p, s = F.fp4_rmsnorm_quant(x, gamma, grid("e4m3"), F.gran("group", 128))
    q, t = F.fp4_rmsnorm_quant(tail, gamma, grid("e4m3"), F.gran("group", 128))
    assert torch.equal(p[-5:], q) and torch.equal(s[-5 * 64:], t)
    assert not p[:-5].any() and not s[:-5 * 64].any()


# ---------------------------------------------------------------- SwiGLU --------------
@pytest.mark.parametrize("rows,cols,xt,fmt,mode,group,f16", [
    (1, 8, "f32", "e4m3", "row", 0, False), (8, 2048, "bf16", "e4m3", "group", 128, False),
    (3, 1416, "bf16", "e5m2", "group", 128, True), (77, 344, "bf16", "e4m3", "row", 0, False),
    (5, 13824, "f32", "e4m3", "group", 512, False), (2, 65536, "bf16", "e5m2", "row", 0, True),
    (130, 4104, "bf16", "e4m3", "tensor", 0, False), (2050, 136, "bf16", "e4m3", "group", 8, False),
    (257, 2080, "f32", "e4m3", "group", 64, False)])
def test_swiglu(rows, cols, xt, fmt, mode, group, f16):
    say("swiglu", rows, cols, xt, fmt, mode, group)
    g = rng(rows + cols)
    x = 3 * randn(g, rows, 2 * cols)
    x[:, ::7] *= 12  # gates far out on both sides
    x[rows // 2] = 0
    x = x.to(TYPES[xt])
    scale = torch.tensor([8.0 / QMAX[fmt]]) if mode == "tensor" else None
    shift = -torch.randint(0, 5, (cols,), generator=g).to(torch.int8) if mode == "tensor" else None
    packed, scales = F.fp4_swiglu_quant(x.to(DEV), grid(fmt), F.gran(mode, group, "f16" if f16 else "f32"),
                                        tensor_scale=scale.to(DEV) if scale is not None else None,
                                        col_shift=shift.to(DEV) if shift is not None else None)
    gate, up = x.double().chunk(2, 1)
    h = gate / (1 + torch.exp(-gate)) * up
    err = (2 * gate.abs() + 8) * U * h.abs() + 2.0 ** -100 * up.abs()
    check_codes(fmt, packed, scales, h, err, mode, group, f16, scale, shift)


def test_swiglu_extremes():
    """Gates at the ends of binary32: the limits of SiLU, never NaN."""
    gate = torch.tensor([-3.4e38, -1e30, -200.0, -88.0, -0.0, 0.0, 88.0, 200.0])
    x = torch.cat([gate, torch.ones(8)])[None]
    packed, scales = F.fp4_swiglu_quant(x.to(DEV), grid("e4m3"), F.gran("tensor"), tensor_scale=torch.ones(1, device=DEV))
    got = packed.cpu().view(torch.float8_e4m3fn).float()[0]
    assert got.tolist() == [0, 0, 0, 0, 0, 0, 88.0, 208.0] or got.tolist() == [0, 0, 0, 0, 0, 0, 88.0, 192.0]


# ---------------------------------------------------------------- weights -------------
@pytest.mark.parametrize("batch,n,k,wt,fmt", [(None, 128, 128, "f32", "e4m3"), (None, 1, 8, "f32", "e4m3"),
                                              (None, 300, 520, "bf16", "e5m2"), (3, 131, 1096, "bf16", "e4m3"),
                                              (2, 257, 136, "f32", "e5m2")])
def test_quantize_block(batch, n, k, wt, fmt):
    """Bit for bit: exact maxima, the same binary32 divisions, the nearest codes."""
    say("quantize_block", batch, n, k, wt, fmt)
    g = rng(n + k)
    w = 0.02 * randn(g, batch or 1, n, k)
    w[:, :1] *= 30
    if n > 128:
        w[:, 128:] = 0  # a block of zeros
    w = w.to(TYPES[wt])
    packed, scales = F.fp4_quantize_block((w if batch else w[0]).to(DEV), grid(fmt))
    packed, scales = packed.cpu().view(-1, n, k), scales.cpu().view(-1, -(-n // 128), -(-k // 128))
    og = O.fp8(*GRIDS[fmt])
    for b in range(batch or 1):
        for i in range(0, n, 128):
            for j in range(0, k, 128):
                v = w[b, i:i + 128, j:j + 128].float().numpy()
                s = np.float32(np.abs(v).max()) / np.float32(QMAX[fmt])
                assert scales[b, i // 128, j // 128].item() == s
                r = np.float32(0) if s == 0 else np.float32(1) / s
                assert np.array_equal(packed[b, i:i + 128, j:j + 128].numpy(), O.quantize(v, r, og).astype(np.uint8))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_conversion_of_every_bf16_value(fmt):
    """With a block maximum of Qmax the scale is 1: the codes of all bf16 values in range are
    the oracle's nearest codes (ties to even, subnormals, signed zeros)."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    v = bits[torch.isfinite(bits) & (bits.abs() <= QMAX[fmt])]
    w = torch.zeros(128, 128 * (-(-len(v) // (128 * 127))))
    w[0] = QMAX[fmt]
    body = torch.zeros(127 * w.shape[1])
    body[:len(v)] = v
    w[1:] = body.view(127, -1)
    packed, scales = F.fp4_quantize_block(w.to(DEV), grid(fmt))
    assert (scales == 1).all()
    want = O.quantize(w.numpy(), np.float32(1), O.fp8(*GRIDS[fmt])).astype(np.uint8)
    assert np.array_equal(packed.cpu().numpy(), want)


# ---------------------------------------------------------------- products ------------
def operand(g, rows, K, name, lead=()):
    """Random codes with a spread of magnitudes, and their values."""
    v = (randn(g, *lead, rows, K) * 20).clamp(-QMAX[name], QMAX[name]).to(FLOAT8[name])
    return v.view(torch.uint8), v.double()


def product_reference(av, sa, wv, sw):
    """Exact value and the product over magnitudes; av [M, K], wv [N, K] in 64 bits."""
    K, N = av.shape[1], wv.shape[0]
    a = av * sa.double().repeat_interleave(128, 1)[:, :K]
    w = wv * sw.double().repeat_interleave(128, 1)[:, :K].repeat_interleave(128, 0)[:N]
    return a @ w.t(), a.abs() @ w.abs().t()


def check_product(y, ref, S, K):
    bound = ((2 * K + 2 * -(-K // 128) + 4) * U + 7 * 2.0 ** -13) * S
    got = y.cpu().double()
    if y.dtype == torch.bfloat16:
        bound = bound * 1.01 + 2.0 ** -8 * ref.abs()
    d = (got - ref).abs()
    used = (d / bound.clamp_min(1e-300)).max().item() if d.numel() else 0.0
    norm = (d.norm() / ref.norm().clamp_min(1e-300)).item()
    say(f"  {used:.3f} of the bound, {norm:.2e} in norm")
    assert used <= 1.0
    assert norm <= (1e-3 if y.dtype == torch.float32 else 4e-3)


def scales_of(g, *shape):
    """Positive, over several binades, some zero."""
    s = torch.exp2(3 * randn(g, *shape)) * 1e-3
    s[torch.rand(shape, generator=g) < 0.02] = 0.0
    return s


PRODUCT = [(M, N, K) for M, N, K in [
    (1, 1, 16), (1, 128, 128), (1, 11008, 4096), (2, 130, 144), (5, 4096, 272), (16, 257, 5120), (17, 64, 1040), (31, 1000, 528),
    (33, 96, 4112), (64, 4100, 2080), (65, 131, 160), (127, 128, 384), (128, 256, 512), (129, 513, 1296), (200, 300, 2064),
    (255, 1024, 640), (257, 259, 272), (300, 4100, 1040), (512, 512, 128), (777, 1025, 400), (1024, 2304, 2048), (2049, 200, 144)]]


@pytest.mark.parametrize("M,N,K", PRODUCT)
def test_product(M, N, K):
    say("product", M, N, K)
    g = rng(M * 7 + N * 3 + K)
    a, av = operand(g, M, K, "e4m3")
    w, wv = operand(g, N, K, "e4m3")
    sa, sw = scales_of(g, M, -(-K // 128)), scales_of(g, -(-N // 128), -(-K // 128))
    ref, S = product_reference(av, sa, wv, sw)
    args = [t.to(DEV) for t in (a, sa, w, sw)]
    y = F.fp4_gemm_block(*args, grid("e4m3"), grid("e4m3"), y_dtype=torch.float32)
    check_product(y, ref, S, K)
    yb = F.fp4_gemm_block(*args, grid("e4m3"), grid("e4m3"))
    assert torch.equal(yb, y.bfloat16())
    assert torch.equal(y, F.fp4_gemm_block(*args, grid("e4m3"), grid("e4m3"), y_dtype=torch.float32))


@pytest.mark.parametrize("fa,fw", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M,N,K", [(3, 200, 400), (70, 300, 272), (300, 520, 1040)])
def test_product_formats(M, N, K, fa, fw):
    say("product", M, N, K, fa, fw)
    g = rng(M + N + K)
    a, av = operand(g, M, K, fa)
    w, wv = operand(g, N, K, fw)
    sa, sw = scales_of(g, M, -(-K // 128)), scales_of(g, -(-N // 128), -(-K // 128))
    ref, S = product_reference(av, sa, wv, sw)
    y = F.fp4_gemm_block(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), grid(fa), grid(fw), y_dtype=torch.float32)
    check_product(y, ref, S, K)


@pytest.mark.parametrize("M", [1, 30, 150, 400])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_product_strides(M, dtype):
    """Operands, scales and output inside wider matrices; odd output rows; nothing outside is
    read or written (the outside holds NaN codes and values)."""
    say("product strides", M, dtype)
    N, K = 203, 336
    g = rng(M)
    a, av = operand(g, M, K, "e4m3")
    w, wv = operand(g, N, K, "e4m3")
    sa, sw = scales_of(g, M, 3), scales_of(g, 2, 3)
    ref, S = product_reference(av, sa, wv, sw)

    def inside(t, extra, fill):
        b = torch.full((t.shape[0] + 3, t.shape[1] + extra), fill, dtype=t.dtype)
        b[:t.shape[0], :t.shape[1]] = t
        return b.to(DEV)[:t.shape[0], :t.shape[1]]
    y = torch.full((M + 2, N + 6), 5.0, dtype=dtype, device=DEV)
    F.fp4_gemm_block(inside(a, 48, 0x7f), inside(sa, 2, math.nan), inside(w, 16, 0x7f), inside(sw, 5, math.nan), grid("e4m3"),
                     grid("e4m3"), y=y[:M, :N])
    check_product(y[:M, :N], ref, S, K)
    assert (y[M:] == 5).all() and (y[:, N:] == 5).all()


def device_operand(g, rows, K, name, lead=()):
    """As operand(), on the GPU."""
    v = (torch.randn(*lead, rows, K, device=DEV, generator=g) * 20).clamp(-QMAX[name], QMAX[name]).to(FLOAT8[name])
    return v.view(torch.uint8), v.double()


def device_scales(g, *shape):
    s = torch.exp2(3 * torch.randn(*shape, device=DEV, generator=g)) * 1e-3
    return s.masked_fill(torch.rand(*shape, device=DEV, generator=g) < 0.02, 0.0)


# Long K (several chunks of scales, a cut last block) on each kernel and tile size, every output
# checked; the reference in 64 bits on the GPU.
@pytest.mark.parametrize("M,N,K", [(5, 300, 7184), (16, 5000, 2576), (14, 9700, 3344), (90, 500, 7184), (1500, 2300, 2832),
                                   (1900, 2500, 2576), (3000, 3100, 3344), (2100, 4400, 1168)])
def test_product_large(M, N, K):
    say("product large", M, N, K)
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    a, av = device_operand(g, M, K, "e4m3")
    w, wv = device_operand(g, N, K, "e4m3")
    sa, sw = device_scales(g, M, -(-K // 128)), device_scales(g, -(-N // 128), -(-K // 128))
    ref, S = product_reference(av, sa, wv, sw)
    y = F.fp4_gemm_block(a, sa, w, sw, grid("e4m3"), grid("e4m3"), y_dtype=torch.float32)
    check_product(y, ref.cpu(), S.cpu(), K)
    for _ in range(3):
        assert torch.equal(F.fp4_gemm_block(a, sa, w, sw, grid("e4m3"), grid("e4m3")), y.bfloat16())


@pytest.mark.parametrize("M,N,K", [(70, 200, 1040), (300, 328, 272), (1030, 1000, 400), (4100, 2056, 144), (4200, 4104, 272)])
def test_product_wide_rows(M, N, K):
    """bf16 rows that take 16-byte stores, with a cut last piece: equal to the rounded f32 rows,
    nothing written past them, on each tile size."""
    say("product wide rows", M, N, K)
    g = torch.Generator(device=DEV)
    g.manual_seed(M)
    a = (torch.randn(M, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
    w = (torch.randn(N, K, device=DEV, generator=g) * 20).to(torch.float8_e4m3fn).view(torch.uint8)
    sa, sw = torch.rand(M, -(-K // 128), device=DEV, generator=g), torch.rand(-(-N // 128), -(-K // 128), device=DEV, generator=g)
    for n in (N, N - 3):
        f = F.fp4_gemm_block(a, sa, w[:n], sw[:-(-n // 128)], grid("e4m3"), grid("e4m3"), y_dtype=torch.float32)
        y = torch.full((M + 1, N + 24), 5.0, dtype=torch.bfloat16, device=DEV)
        F.fp4_gemm_block(a, sa, w[:n], sw[:-(-n // 128)], grid("e4m3"), grid("e4m3"), y=y[:M, :n])
        assert torch.equal(y[:M, :n], f.bfloat16())
        assert (y[M:] == 5).all() and (y[:, n:] == 5).all()


def test_product_past_32_bits():
    """Operands, and an output, of more than 2 GiB."""
    for M, N, K in ((560000, 40, 4096), (40, 560000, 4096), (70000, 33000, 128)):
        say("product", M, N, K)
        a = torch.zeros(M, K, dtype=torch.uint8, device=DEV)
        w = torch.zeros(N, K, dtype=torch.uint8, device=DEV)
        kb = K // 128
        g = rng(M)
        at, avt = operand(g, 40, K, "e4m3")
        wt, wvt = operand(g, 40, K, "e4m3")
        a[-40:], w[-40:] = at.to(DEV), wt.to(DEV)
        sa = torch.ones(M, kb, device=DEV)
        sw = torch.ones(-(-N // 128), kb, device=DEV)
        y = F.fp4_gemm_block(a, sa, w, sw, grid("e4m3"), grid("e4m3"))
        ref, S = product_reference(avt, torch.ones(40, kb), wvt, torch.ones(1, kb))
        check_product(y[-40:, -40:], ref, S, K)
        if M > 40:
            assert not y[:-40].any()
        del a, w, y


def test_product_of_the_quantizers_outputs():
    """Codes and scales as the norm and the weight quantizer leave them."""
    g = rng(3)
    x, w = randn(g, 50, 528).bfloat16().to(DEV), (0.02 * randn(g, 260, 528)).to(DEV)
    a, sa = F.fp4_rmsnorm_quant(x, torch.ones(528, device=DEV), grid("e4m3"), F.gran("group", 128))
    wq, sw = F.fp4_quantize_block(w, grid("e4m3"))
    y = F.fp4_gemm_block(a, sa, wq, sw, grid("e4m3"), grid("e4m3"), y_dtype=torch.float32)
    xn = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    want = (xn @ w.double().t()).cpu()
    assert ((y.cpu().double() - want).norm() / want.norm()) < 0.05  # two 3-bit mantissas


# ---------------------------------------------------------------- routing -------------
def route_reference(logits, top_k, score, bias, groups, top_groups, group_top, renormalise, scale):
    """Per token, in 64 bits, by sorting (key, -index)."""
    L = logits.double().numpy()
    T, E = L.shape
    idx, wgt = np.full((T, top_k), -1, np.int32), np.zeros((T, top_k))
    spread = np.zeros(T)
    for t in range(T):
        use = [e for e in range(E) if np.isfinite(L[t, e])]
        if not use:
            continue
        l = np.array([L[t, e] for e in use])
        spread[t] = np.abs(l - (l.max() if score == "softmax" else 0)).max()
        if score == "softmax":
            p = np.exp(l - l.max())
            p /= p.sum()
        else:
            with np.errstate(over="ignore"):
                p = 1 / (1 + np.exp(-l))
        s = dict(zip(use, p))
        key = {e: s[e] + (float(bias[e]) if bias is not None else 0.0) for e in use}
        if groups > 1:
            size = E // groups
            val = {}
            for e in use:
                val.setdefault(e // size, []).append(key[e])
            val = {q: sum(sorted(v, reverse=True)[:group_top]) for q, v in val.items()}
            keep = sorted(val, key=lambda q: (-val[q], q))[:top_groups]
            use = [e for e in use if e // size in keep]
        chosen = sorted(use, key=lambda e: (-key[e], e))[:top_k]
        w = np.array([s[e] for e in chosen])
        if renormalise:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        idx[t, :len(chosen)] = chosen
        wgt[t, :len(chosen)] = w * scale
    flat = np.where(idx.reshape(-1) < 0, E, idx.reshape(-1))
    slots = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[slots], np.arange(E + 1))
    return idx, wgt, offsets, slots, spread


def coarse_logits(g, T, E, score, biased):
    """Logits whose keys cannot be turned round by rounding: keys that are equal are equal for
    equal logits (and biases), all others differ by more than 1e-5."""
    if not biased:
        return torch.randint(-40, 41, (T, E), generator=g).float() / 16, None
    if score == "softmax":
        # scores of equal logits: keys differ by the bias alone
        return torch.full((T, E), 0.5), torch.randperm(E, generator=g).float() / 64
    # scores are 1/2 or below 1e-13; biases on a grid of distinct values with distinct pair sums
    l = torch.where(torch.rand(T, E, generator=g) < 0.5, 0.0, -32.0)
    return l, torch.rand(E, generator=g) * 8


def check_routing(got, want, E):
    idx, wgt, offsets, slots, spread = want
    assert np.array_equal(got.experts.cpu().numpy(), idx)
    w = got.weights.cpu().numpy().astype(np.float64)
    assert (np.abs(w - wgt) <= (2 * spread[:, None] + 40) * U * np.abs(wgt) + 1e-37).all()
    if got.offsets is not None:
        assert np.array_equal(got.offsets.cpu().numpy(), offsets)
        assert np.array_equal(got.slots.cpu().numpy(), slots)


@pytest.mark.parametrize("T,E,k,score,biased,groups,top_groups,group_top,renorm,dtype", [
    (1, 1, 1, "softmax", False, 1, 1, 1, True, "f32"), (1, 64, 6, "softmax", False, 1, 1, 1, True, "f32"),
    (3, 8, 2, "sigmoid", True, 1, 1, 1, False, "bf16"), (200, 60, 4, "softmax", False, 1, 1, 1, False, "bf16"),
    (65, 160, 8, "softmax", False, 8, 3, 1, False, "f32"), (130, 256, 8, "sigmoid", True, 8, 4, 2, True, "f32"),
    (77, 384, 8, "softmax", True, 1, 1, 1, True, "f32"), (40, 1024, 32, "softmax", False, 64, 9, 2, True, "f32"),
    (33, 1000, 5, "sigmoid", False, 1, 1, 1, True, "bf16"), (500, 128, 8, "sigmoid", True, 4, 2, 2, True, "f32"),
    (5000, 16, 2, "softmax", False, 1, 1, 1, True, "f32"), (2500, 72, 6, "sigmoid", True, 9, 4, 2, True, "f32"),
    (300, 96, 3, "softmax", True, 32, 5, 2, True, "f32"), (150, 512, 8, "sigmoid", True, 16, 4, 2, True, "f32"),
    (700, 64, 8, "sigmoid", False, 64, 8, 1, False, "f32"), (90, 33, 32, "softmax", False, 1, 1, 1, True, "f32"),
    (50, 700, 8, "softmax", False, 1, 1, 1, True, "f32"), (45, 768, 6, "sigmoid", True, 1, 1, 1, True, "bf16"),
    (20, 1023, 8, "softmax", False, 33, 5, 1, True, "f32"), (120, 192, 8, "sigmoid", True, 8, 3, 2, True, "f32")])
def test_route(T, E, k, score, biased, groups, top_groups, group_top, renorm, dtype):
    say("route", T, E, k, score, biased, groups, top_groups, group_top)
    g = rng(T + E)
    l, bias = coarse_logits(g, T, E, score, biased)
    if T > 2:
        for v in (-math.inf, math.inf, math.nan):
            l[torch.rand(T, E, generator=g) < 0.03] = v
        l[T // 2] = -math.inf  # a padding token
        l[T // 3, 1:] = -math.inf  # fewer usable than top_k
        l[T // 4] = math.nan
    l = l.to(TYPES[dtype])
    got = F.fp4_route(l.to(DEV), k, score=score, bias=bias.to(DEV) if bias is not None else None, groups=groups,
                      top_groups=top_groups, group_top=group_top, renormalise=renorm, scale=2.5)
    check_routing(got, route_reference(l.float(), k, score, bias, groups, top_groups, group_top, renorm, 2.5), E)
    again = F.fp4_route(l.to(DEV), k, score=score, bias=bias.to(DEV) if bias is not None else None, groups=groups,
                        top_groups=top_groups, group_top=group_top, renormalise=renorm, scale=2.5, layout=False)
    assert torch.equal(again.experts, got.experts) and torch.equal(again.weights, got.weights) and again.slots is None


def test_route_extremes():
    """Logits at the ends of the type: finite values are usable, scores may vanish."""
    top = torch.finfo(torch.float32).max
    l = torch.tensor([[-top, -top, -top, -top], [top, 0.0, -top, top], [-top, 3.0, -top, 1.0], [200.0, -200.0, 0.0, -top]])
    for score in ("softmax", "sigmoid"):
        got = F.fp4_route(l.to(DEV), 3, score=score, renormalise=True)
        check_routing(got, route_reference(l, 3, score, None, 1, 1, 1, True, 1.0), 4)


def test_route_strided_and_empty():
    g = rng(2)
    l = torch.randint(-40, 41, (50, 70), generator=g).float().div(16).to(DEV)
    a, b = F.fp4_route(l[:, 3:64], 4), F.fp4_route(l[:, 3:64].contiguous(), 4)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    r = F.fp4_route(torch.empty(0, 16, device=DEV), 2)
    assert r.experts.shape == (0, 2) and not r.offsets.any() and r.slots.numel() == 0


@pytest.mark.parametrize("T,E,k", [(257, 8, 2), (2048, 256, 8), (40000, 64, 8), (300000, 8, 4), (16, 1024, 8), (33, 5, 5)])
def test_route_layout(T, E, k):
    """The layout of many slots, skewed so that one expert takes most and some take none."""
    say("layout", T, E, k)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    l = torch.randn(T, E, device=DEV, generator=g)
    l[:, 0] += 3
    l[:, E // 2] = -math.inf
    l[::97] = math.nan
    r = F.fp4_route(l, k)
    flat = r.experts.view(-1).long()
    flat = torch.where(flat < 0, E, flat)
    slots = torch.sort(flat, stable=True).indices
    assert torch.equal(r.slots.long(), slots)
    assert torch.equal(r.offsets.long(), torch.searchsorted(flat[slots], torch.arange(E + 1, device=DEV)))


# ---------------------------------------------------------------- experts -------------
EXPERTS = [
    # slots per row, rows, experts, top_k, N, K, skew
    (1, 1, 8, 2, 130, 272, 0), (2, 1, 8, 2, 64, 144, 0), (8, 8, 64, 8, 256, 1040, 0), (4, 40, 60, 4, 200, 400, 1),
    (1, 33, 16, 2, 513, 640, 0), (2, 300, 4, 2, 300, 528, 1), (8, 257, 8, 8, 129, 272, 0), (6, 150, 100, 6, 96, 144, 2),
    (2, 1025, 3, 2, 260, 384, 2), (1, 600, 1, 1, 384, 512, 0), (8, 700, 40, 8, 520, 256, 1)]


@pytest.mark.parametrize("per,rows,E,k,N,K,skew", EXPERTS)
def test_experts(per, rows, E, k, N, K, skew):
    say("experts", per, rows, E, k, N, K, skew)
    g = rng(rows + E + N)
    l = randn(g, rows, E)
    if skew:
        l[:, 0] += 4  # one long list
        l[:, E - 1] = -math.inf  # an expert without slots
    if skew == 2:
        l[rows // 2:rows // 2 + 3] = -math.inf  # tokens without experts
    r = F.fp4_route(l.to(DEV), k)
    S = rows * k
    arows = rows if per == k else S
    a, av = operand(g, arows, K, "e4m3")
    w, wv = operand(g, N, K, "e4m3", (E,))
    sa, sw = scales_of(g, arows, -(-K // 128)), scales_of(g, E, -(-N // 128), -(-K // 128))
    y = torch.full((S, N), 7.0, device=DEV)
    args = (a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), grid("e4m3"), grid("e4m3"), r.offsets, r.slots)
    F.fp4_gemm_experts(*args, slots_per_row=k if per == k else 1, y=y)
    choice = r.experts.view(-1).cpu()
    got = y.cpu()
    for e in range(E):
        s = torch.nonzero(choice == e).view(-1)
        if len(s):
            src = s // k if per == k else s
            ref, S_ = product_reference(av[src], sa[src], wv[e], sw[e])
            check_product(got[s], ref, S_, K)
    assert (got[choice < 0] == 7).all()
    yb = torch.full((S, N), 7.0, dtype=torch.bfloat16, device=DEV)
    F.fp4_gemm_experts(*args, slots_per_row=k if per == k else 1, y=yb)
    assert torch.equal(yb, y.bfloat16())


# Lists from empty to long on each kernel and tile size, long K.
@pytest.mark.parametrize("T,E,k,N,K,shared", [(2, 40, 6, 500, 2576, True), (30, 24, 4, 700, 2576, False), (200, 12, 3, 1300, 2832, True),
                                              (1000, 8, 2, 2500, 2576, True), (2000, 6, 2, 3000, 1168, False),
                                              (3000, 10, 3, 2000, 2576, True)])
def test_experts_large(T, E, k, N, K, shared):
    say("experts large", T, E, k, N, K)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    l = torch.randn(T, E, device=DEV, generator=g) + torch.randn(E, device=DEV, generator=g)
    l[:, 1] = -math.inf
    l[::50] = math.nan
    r = F.fp4_route(l, k)
    rows = T if shared else T * k
    a, av = device_operand(g, rows, K, "e4m3")
    w, wv = device_operand(g, N, K, "e4m3", (E,))
    sa, sw = device_scales(g, rows, -(-K // 128)), device_scales(g, E, -(-N // 128), -(-K // 128))
    y = torch.full((T * k, N), 7.0, device=DEV)
    F.fp4_gemm_experts(a, sa, w, sw, grid("e4m3"), grid("e4m3"), r.offsets, r.slots, slots_per_row=k if shared else 1, y=y)
    choice = r.experts.view(-1)
    for e in range(E):
        s = torch.nonzero(choice == e).view(-1)
        if len(s):
            src = s // k if shared else s
            ref, S_ = product_reference(av[src], sa[src], wv[e], sw[e])
            check_product(y[s], ref.cpu(), S_.cpu(), K)
    assert (y[choice < 0] == 7).all()
    for _ in range(3):
        yb = torch.full((T * k, N), 7.0, dtype=torch.bfloat16, device=DEV)
        F.fp4_gemm_experts(a, sa, w, sw, grid("e4m3"), grid("e4m3"), r.offsets, r.slots, slots_per_row=k if shared else 1, y=yb)
        assert torch.equal(yb, y.bfloat16())


def test_experts_formats_and_strides():
    g = rng(9)
    E, N, K, S = 5, 70, 160, 90
    a, av = operand(g, S, K, "e5m2")
    w, wv = operand(g, N, K, "e5m2", (E,))
    sa, sw = scales_of(g, S, 2), scales_of(g, E, 1, 2)
    choice = torch.randint(0, E, (S,), generator=g)
    slots = torch.sort(choice, stable=True).indices.int().to(DEV)
    offsets = torch.searchsorted(choice.sort().values, torch.arange(E + 1)).int().to(DEV)
    wide = torch.full((E, N + 2, K + 32), 0x7f, dtype=torch.uint8, device=DEV)
    wide[:, :N, :K] = w.to(DEV)
    y = torch.full((S, N + 3), 5.0, device=DEV)
    F.fp4_gemm_experts(a.to(DEV), sa.to(DEV), wide[:, :N, :K], sw.to(DEV), grid("e5m2"), grid("e5m2"), offsets, slots, y=y[:, :N])
    for e in range(E):
        s = torch.nonzero(choice == e).view(-1)
        ref, S_ = product_reference(av[s], sa[s], wv[e], sw[e])
        check_product(y.cpu()[s, :N], ref, S_, K)
    assert (y[:, N:] == 5).all()


def test_experts_ignore_slots_out_of_range():
    """A layout that names slots outside the output writes nothing there and reads no row."""
    g = rng(4)
    N, K, S = 64, 128, 6
    a, av = operand(g, S, K, "e4m3")
    w, wv = operand(g, N, K, "e4m3", (2,))
    slots = torch.tensor([0, -1, 2, 1 << 30, 4, 6], dtype=torch.int32, device=DEV)
    offsets = torch.tensor([-3, 4, 900], dtype=torch.int32, device=DEV)
    y = torch.full((S, N), 5.0, device=DEV)
    F.fp4_gemm_experts(a.to(DEV), torch.ones(S, 1, device=DEV), w.to(DEV), torch.ones(2, 1, 1, device=DEV), grid("e4m3"),
                       grid("e4m3"), offsets, slots, y=y)
    one = torch.ones(1, 1)
    for s, e in ((0, 0), (2, 0), (4, 1)):
        ref, S_ = product_reference(av[s:s + 1], one, wv[e], one)
        check_product(y.cpu()[s:s + 1], ref, S_, K)
    assert (y[[1, 3, 5]] == 5).all()


# ---------------------------------------------------------------- together ------------
def layer_inputs(T=70, D=512, I=256, E=16, k=4, seed=1):
    g = rng(seed)
    t = lambda v: v.to(DEV)  # noqa: E731
    wg, sg = F.fp4_quantize_block(t(0.05 * randn(g, E, 2 * I, D)), grid("e4m3"))
    wd, sd = F.fp4_quantize_block(t(0.05 * randn(g, E, D, I)), grid("e4m3"))
    return dict(x=t(randn(g, T, D).bfloat16()), residual=t(randn(g, T, D).bfloat16()), gamma=t(torch.ones(D)),
                router=t(0.1 * randn(g, D, E)), wg=wg, sg=sg, wd=wd, sd=sd, k=k)


def layer(v):
    """Norm, routing, both expert products, and the experts' outputs joining the stream."""
    e4, g128 = grid("e4m3"), F.gran("group", 128)
    stream, y = torch.empty_like(v["residual"]), torch.empty_like(v["residual"])
    a, sa = F.fp4_rmsnorm_quant(v["x"], v["gamma"], e4, g128, residual=v["residual"], residual_out=stream, y=y)
    r = F.fp4_route(y.float() @ v["router"], v["k"], score="sigmoid")
    gu = F.fp4_gemm_experts(a, sa, v["wg"], v["sg"], e4, e4, r.offsets, r.slots, slots_per_row=v["k"])
    h, sh = F.fp4_swiglu_quant(gu, e4, g128)
    out = F.fp4_gemm_experts(h, sh, v["wd"], v["sd"], e4, e4, r.offsets, r.slots)
    F.fp4_rmsnorm_quant(out, v["gamma"], e4, g128, residual=stream, residual_out=stream, terms=v["k"], term_weights=r.weights)
    return stream


def layer_reference(v):
    h = v["x"].double() + v["residual"].double()
    n = h / (h.square().mean(1, keepdim=True) + 1e-6).sqrt()
    p = torch.sigmoid(n @ v["router"].double())
    w, idx = p.topk(v["k"], 1)
    w = w / w.sum(1, keepdim=True)

    def values(q, s):
        s = s.double().repeat_interleave(128, 1).repeat_interleave(128, 2)
        return q.view(torch.float8_e4m3fn).double() * s[:, :q.shape[1], :q.shape[2]]
    wg, wd = values(v["wg"], v["sg"]), values(v["wd"], v["sd"])
    for j in range(v["k"]):
        gate, up = torch.bmm(wg[idx[:, j]], n[:, :, None])[:, :, 0].chunk(2, 1)
        h = h + w[:, j:j + 1] * torch.bmm(wd[idx[:, j]], (torch.nn.functional.silu(gate) * up)[:, :, None])[:, :, 0]
    return h


def test_expert_layer():
    """The whole layer against 64 bits with the same weights: 8-bit activations (3 mantissa
    bits, 2^-4 / sqrt 3 relative per value) enter twice."""
    v = layer_inputs()
    got, want = layer(v).double(), layer_reference(v)
    delta = want - (v["x"].double() + v["residual"].double())
    err = ((got - want).norm() / delta.norm()).item()
    say(f"  expert layer: {err:.3f} of the update in norm")
    assert err < 0.15


def test_other_stream_and_graph():
    """The same results on a side stream, and from replays of a captured graph."""
    v = layer_inputs(seed=2)
    want = layer(v)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(v)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(v)
    for seed in (3, 4, 5):
        new = layer_inputs(seed=seed)
        for name in ("x", "residual"):
            v[name].copy_(new[name])
        want = layer(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        want = layer(v)
        graph.replay()
        assert torch.equal(out, want)


def test_binding_refusals():
    e4 = grid("e4m3")
    x, w = torch.zeros(4, 256, device=DEV), torch.zeros(8, 256, dtype=torch.uint8, device=DEV)
    one = torch.ones(256, device=DEV)
    with pytest.raises(ValueError):
        F.fp4_rmsnorm_quant(x, one, e4, F.gran("row"), terms=3)
    with pytest.raises(ValueError):
        F.fp4_rmsnorm_quant(x, one[:128], e4, F.gran("row"))
    with pytest.raises(ValueError):
        F.fp4_rmsnorm_quant(x.t(), torch.ones(4, device=DEV), e4, F.gran("row"))
    with pytest.raises(TypeError):
        F.fp4_rmsnorm_quant(x.half(), one, e4, F.gran("row"))
    with pytest.raises(F.FP4Error):
        F.fp4_rmsnorm_quant(x, one, F.grid_minifloat(2, 1), F.gran("row"))
    with pytest.raises(ValueError):
        F.fp4_gemm_block(w, torch.ones(8, 1, device=DEV), w, torch.ones(1, 2, device=DEV), e4, e4)
    with pytest.raises(ValueError):
        F.fp4_gemm_block(w, torch.ones(8, 2, device=DEV), w, torch.ones(1, 2), e4, e4)
    with pytest.raises(ValueError):
        F.fp4_route(x, 4, score="tanh")
    with pytest.raises(F.FP4Error):
        F.fp4_route(x, 64)
    with pytest.raises(ValueError):
        F.fp4_route(x, 4, bias=one.double())
    with pytest.raises(ValueError):
        F.fp4_gemm_experts(w, torch.ones(8, 2, device=DEV), w[None], torch.ones(1, 1, 2, device=DEV), e4, e4,
                           torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(8, dtype=torch.int32, device=DEV))
