"""The norm's and SwiGLU's codes where the rest of the library reads them: the same bits as
fp4_quantize_pack's, decoded by fp4_dequantize, and as operands of fp4_gemm (a scale per token;
a static scale with shifted channels)."""
import pytest
import torch

from test_gpu_layer import F, FLOAT8, check_product, grid, say

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


def randn(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("mode,group,f16", [("row", 0, False), ("row", 0, True), ("group", 8, False), ("group", 64, True),
                                            ("group", 128, False), ("group", 512, False)])
def test_norm_codes_are_the_quantizers(fmt, mode, group, f16):
    """Bit for bit, over as many scales as there are units (2.6 million with groups of 8): the
    normed rows come out in binary32 and go through fp4_quantize_pack."""
    rows, cols = 40000, 512
    say("norm codes", fmt, mode, group, f16)
    x = randn(1, rows, cols) * torch.exp2(4 * randn(2, rows, 1))
    gamma = torch.exp2(3 * randn(3, cols))
    gr, y = F.gran(mode, group, "f16" if f16 else "f32"), torch.empty(rows, cols, device=DEV)
    p, s = F.fp4_rmsnorm_quant(x, gamma, grid(fmt), gr, y=y)
    q, t = F.fp4_quantize_pack(y, grid(fmt), gr)
    assert torch.equal(s, t.view(-1)) and torch.equal(p, q)
    d = F.fp4_dequantize(p, grid(fmt), gr, s)
    width = cols if mode == "row" else group
    assert torch.equal(d, p.view(FLOAT8[fmt]).float() * s.float().view(rows, -1).repeat_interleave(width, 1))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_static_codes_are_the_quantizers(fmt):
    rows, cols = 3000, 520
    say("static codes", fmt)
    x, gamma = randn(4, rows, cols), torch.exp2(3 * randn(5, cols))
    scale = torch.full((1,), 0.0123, device=DEV)
    shift = -torch.randint(0, 65, (cols,), device=DEV).to(torch.int8)
    for k in (None, shift):
        y = torch.empty(rows, cols, device=DEV)
        p, _ = F.fp4_rmsnorm_quant(x, gamma, grid(fmt), F.gran("tensor"), tensor_scale=scale, col_shift=k, y=y)
        q, _ = F.fp4_quantize_pack(y, grid(fmt), F.gran("tensor"), tensor_scale=scale, col_shift=k)
        assert torch.equal(p, q)


@pytest.mark.parametrize("fa,fw", [("e4m3", "e4m3"), ("e5m2", "e5m2"), ("e4m3", "e5m2")])
@pytest.mark.parametrize("M,N,K", [(1, 300, 544), (70, 256, 512), (300, 520, 1056)])
def test_tokens_scales_in_the_product(M, N, K, fa, fw):
    """Codes with a scale per token, from the norm and from SwiGLU, through fp4_gemm: against the
    decoded operands in 64 bits, the bound of packed products."""
    say("per token", M, N, K, fa, fw)
    w, sw = F.fp4_quantize_pack(0.02 * randn(6, N, K), grid(fw), F.gran("row"))
    wv = w.view(FLOAT8[fw]).double() * sw.double().view(N, 1)
    for a, sa in (F.fp4_rmsnorm_quant(randn(7, M, K), torch.ones(K, device=DEV), grid(fa), F.gran("row")),
                  F.fp4_swiglu_quant(randn(8, M, 2 * K), grid(fa), F.gran("row"))):
        y = F.fp4_gemm(a, w, sw, grid(fw), F.gran("row"), a_grid=grid(fa), a_scale=sa, a_scale_mode="row", y_dtype=torch.float32)
        av = a.view(FLOAT8[fa]).double() * sa.double().view(M, 1)
        check_product(y, (av @ wv.t()).cpu(), (av.abs() @ wv.abs().t()).cpu(), K)


@pytest.mark.parametrize("M", [5, 200])
def test_static_scale_in_the_product(M):
    """Pre-shifted weights, and the norm's codes with the static scale and shifts that belong to
    them: against the decoded operands in 64 bits."""
    N, K = 264, 512
    say("static", M)
    e4 = grid("e4m3")
    gamma = torch.exp2(2 * randn(9, K))
    x = randn(10, 500, K)
    n = torch.empty(500, K, device=DEV)
    F.fp4_rmsnorm_quant(x, gamma, y=n)
    shift, scale, w, sw = F.fp4_preshift_weights(0.02 * randn(11, N, K), F.fp4_calibrate(n, "column"), e4, e4, F.gran("row"))
    a, _ = F.fp4_rmsnorm_quant(x[:M], gamma, e4, F.gran("tensor"), tensor_scale=scale, col_shift=shift)
    y = F.fp4_gemm(a, w, sw, e4, F.gran("row"), a_grid=e4, a_scale=scale, y_dtype=torch.float32)
    av, wv = a.view(FLOAT8["e4m3"]).double() * scale.double(), w.view(FLOAT8["e4m3"]).double() * sw.double().view(N, 1)
    check_product(y, (av @ wv.t()).cpu(), (av.abs() @ wv.abs().t()).cpu(), K)
