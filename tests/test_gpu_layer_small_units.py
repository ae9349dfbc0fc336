"""FP8 codes of units whose largest value is tiny: down to binary32's smallest subnormal, with
zeros among the values.

A unit's scale is fl32(amax / Qmax), but no less than 2^-126 unless amax is 0, so its reciprocal
is finite and at most 2^126.  Checked in 64 bits: every code is finite, zeros are zeros, and
code * scale is within half a step of the grid of the value v.  Half a step is at most
max(|v| 2^-(m + 1), s q), q half the smallest code's value; v's product with the reciprocal
(normal wherever v is not 0: 2^-149 2^124 at least) carries two roundings, 2.1 u |v| with
u = 2^-24.  A value known to within err adds err, and 2^-(m + 1) err through its half step.
"""
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
LEAST = {"e4m3": 2.0 ** -9, "e5m2": 2.0 ** -16}  # smallest code


def say(*a):
    print(*a, flush=True)


def grid(name):
    return F.grid_minifloat(*GRIDS[name])


def peaks(fmt):
    """Largest values of units: the ends of the subnormals, and around the scales 2^-128 and
    2^-126 where a reciprocal leaves binary32 and where a scale becomes normal."""
    q = QMAX[fmt]
    return [2.0 ** -149, 3 * 2.0 ** -149, 1e-40, 1e-37, 1e-35, 1e-33, q * 2.0 ** -128, q * 2.0 ** -127, q * 2.0 ** -126,
            q * 2.0 ** -126 * (1 - 2.0 ** -20), q * 2.0 ** -125]


def scale_of(amax, fmt):
    """The scale of units with these largest values (binary32 exactly)."""
    s = np.asarray(amax, np.float32) / np.float32(QMAX[fmt])
    return np.where(np.asarray(amax) > 0, np.maximum(s, np.float32(2.0 ** -126)), np.float32(0))


def check_values(fmt, packed, v, s, err=0.0):
    """Codes of v (64 bits, known to within err) with the scales s, per value."""
    got = packed.cpu().view(FLOAT8[fmt]).double()
    assert torch.isfinite(got).all(), "a code that is no number"
    assert (got[v == 0] == 0).all()
    m = GRIDS[fmt][1]
    step = torch.maximum(v.abs() * 2.0 ** -(m + 1), s * LEAST[fmt] / 2)
    d = (got * s - v).abs()
    assert (d <= step + 2.1 * U * v.abs() + err * (1 + 2.0 ** -(m + 1) + 2.1 * U)).all(), (d / (step + err).clamp_min(1e-300)).max()


def patterns(rows, cols, seed):
    """Signed values of [0.25, 1], a third of them zero, the first of every 8 the largest, 1."""
    g = torch.Generator()
    g.manual_seed(seed)
    v = (0.25 + 0.75 * torch.rand(rows, cols, generator=g)) * torch.where(torch.rand(rows, cols, generator=g) < 0.5, -1.0, 1.0)
    v[torch.rand(rows, cols, generator=g) < 0.33] = 0.0
    v[:, ::8] = 1.0
    return v


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("mode,group", [("row", 0), ("group", 8), ("group", 128)])
def test_norm(fmt, mode, group):
    """Tiny gamma.  The normed rows come out in binary32 beside their codes, so the reference
    needs no error bound: the scale is exact, bit for bit."""
    cols = 264
    for peak in peaks(fmt):
        say("norm", fmt, mode, group, peak)
        x = patterns(5, cols, 1)
        x[3] = 0
        gamma = torch.full((cols,), peak, dtype=torch.float64).float()
        gamma[-100:] = 0  # units of zeros, in binary32 too
        y = torch.empty(5, cols, device=DEV)
        p, s = F.fp4_rmsnorm_quant(x.to(DEV), gamma.to(DEV), grid(fmt), F.gran(mode, group), y=y)
        n = y.cpu()
        assert (n[:, ::8][[0, 1, 2, 4], :20] != 0).all()
        width = cols if mode == "row" else group
        units = -(-cols // width)
        amax = torch.nn.functional.pad(n.abs(), (0, units * width - cols)).view(5, units, width).amax(2).numpy()
        assert np.array_equal(s.cpu().numpy().reshape(5, units), scale_of(amax, fmt))
        check_values(fmt, p, n.double(), s.cpu().double().view(5, units).repeat_interleave(width, 1)[:, :cols])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("mode,group", [("row", 0), ("group", 8), ("group", 128)])
def test_swiglu(fmt, mode, group):
    """Tiny up values beside a gate of 40 (SiLU 40), and gates at -86 and below.  h is within
    (2 |g| + 8) u of its exact value, 2^-100 |u| for gates below -87, and 2^-150 where it is
    subnormal (two products)."""
    cols = 264
    width = cols if mode == "row" else group
    units = -(-cols // width)
    for peak in peaks(fmt):
        say("swiglu", fmt, mode, group, peak)
        up = (patterns(4, cols, 2).double() * max(peak / 32, 2.0 ** -149)).float()
        gate = torch.full((4, cols), 40.0)
        gate[1], up[1] = -86.0 - torch.rand(cols) * 3, patterns(1, cols, 3)[0] * 0.25
        up[2] = 0
        x = torch.cat([gate, up], 1)
        p, s = F.fp4_swiglu_quant(x.to(DEV), grid(fmt), F.gran(mode, group))
        g, u = gate.double(), up.double()
        h = g / (1 + torch.exp(-g)) * u
        err = (2 * g.abs() + 8) * U * h.abs() + torch.where(g < -87, 2.0 ** -100 * u.abs(), 0.0) + 2.0 ** -149
        err[u == 0] = 0
        s64 = s.cpu().double().view(4, units)
        pad = (0, units * width - cols)
        amax = torch.nn.functional.pad(h.abs(), pad).view(4, units, width).amax(2)
        most = torch.nn.functional.pad(err, pad).view(4, units, width).amax(2) / QMAX[fmt]
        want = torch.where(amax > 0, (amax / QMAX[fmt]).clamp_min(2.0 ** -126), 0.0)
        assert ((s64 - want).abs() <= most + want * 2 * U).all()
        check_values(fmt, p, h, s64.repeat_interleave(width, 1)[:, :cols], err)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize_block(fmt, dtype):
    """Bit for bit: the scale, and the oracle's codes of the values times its reciprocal."""
    og = O.fp8(*GRIDS[fmt])
    for peak in peaks(fmt):
        say("quantize_block", fmt, dtype, peak)
        w = (patterns(130, 136, 4).double() * peak).to(dtype)
        w[:128, 128:] = 0
        p, s = F.fp4_quantize_block(w.to(DEV), grid(fmt))
        for i in (0, 128):
            for j in (0, 128):
                v = w[i:i + 128, j:j + 128].float()
                want = scale_of(v.abs().max().item(), fmt)
                got = s[i // 128, j // 128].item()
                assert got == want
                codes = p[i:i + 128, j:j + 128].cpu().contiguous()
                check_values(fmt, codes, v.double(), torch.full_like(v, got, dtype=torch.float64))
                r = np.float32(0) if want == 0 else np.float32(1) / np.float32(want)
                assert np.array_equal(codes.numpy(), O.quantize(v.numpy(), r, og).astype(np.uint8))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("scale,shift", [(2.0 ** -149, None), (1e-39, None), (1e-30, -64), (2.0 ** -70, -64), (2.0 ** -130, -3)])
def test_static_scales(fmt, scale, shift):
    """A given scale (with its shift) whose reciprocal is past binary32: zeros stay zeros, values
    past the grid's end are its end."""
    x = patterns(3, 72, 5)
    k = torch.full((72,), shift, dtype=torch.int8, device=DEV) if shift is not None else None
    ts = torch.tensor([scale], device=DEV)
    p, _ = F.fp4_rmsnorm_quant(x.to(DEV), torch.ones(72, device=DEV), grid(fmt), F.gran("tensor"), tensor_scale=ts, col_shift=k)
    got = p.cpu().view(FLOAT8[fmt]).float()
    assert torch.equal(got, torch.sign(x) * QMAX[fmt])
    x2 = torch.cat([torch.full((3, 72), 40.0), x], 1)
    p, _ = F.fp4_swiglu_quant(x2.to(DEV), grid(fmt), F.gran("tensor"), tensor_scale=ts, col_shift=k)
    assert torch.equal(p.cpu().view(FLOAT8[fmt]).float(), torch.sign(x) * QMAX[fmt])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_products_stay_finite(fmt):
    """Rows and blocks of tiny values through the product: every output is a number."""
    e = grid(fmt)
    x, w = patterns(20, 256, 6), patterns(200, 256, 7)
    gamma = torch.ones(256)
    gamma[:128] = 1e-39
    w[:128] *= 1e-38
    a, sa = F.fp4_rmsnorm_quant(x.to(DEV), gamma.to(DEV), e, F.gran("group", 128))
    wq, sw = F.fp4_quantize_block(w.to(DEV), e)
    y = F.fp4_gemm_block(a, sa, wq, sw, e, e, y_dtype=torch.float32)
    assert torch.isfinite(y).all() and (y[:, 128:] != 0).any()
