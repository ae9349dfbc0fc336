"""The binding of the key/value cache without a GPU, on host tensors: what it has to refuse, and what it
hands to the library for tensors of any layout; no call gets as far as a launch."""
import ctypes

import pytest
import torch

import bit_floating_point_amd as F
from bit_floating_point_amd import _lib as L
from bit_floating_point_amd import cache as C

E4M3, E2M1 = F.grid_minifloat(4, 3), F.grid_minifloat(2, 1)
ROW, F16_ROW, ONE = F.gran("row"), F.gran("row", scale_dtype="f16"), F.gran("tensor")
I32 = torch.int32


@pytest.fixture
def given(monkeypatch):
    """The descriptors that reach the library, as structures."""
    calls = []

    def launch(cache, func, desc, *more):
        kind = C.fp4_attend_desc if func == "fp4_attend" else C.fp4_cache_rows_desc
        calls.append((func, kind.from_buffer_copy(desc), *more))
    monkeypatch.setattr(C, "_launch", launch)
    return calls


@pytest.fixture
def host(monkeypatch):
    """Calls go to the library's host checks, without a stream."""
    monkeypatch.setattr(C, "_launch", lambda cache, func, *a: L.check(C._call(func)(cache.desc, *a, None), func))


def new(pages=6, heads=2, size=16, dim=128, grid=E4M3, g=ROW, **kw):
    return F.kv_cache(pages, heads, size, dim, grid, g, device="cpu", **kw)


def ints(*shape):
    return torch.zeros(*shape, dtype=I32)


def test_new_caches():
    c = new()
    assert c.k.shape == (6, 2, 16, 128) and c.k.dtype == torch.uint8 and c.k_scales.shape == (6, 2, 16) and c.k_scales.dtype == torch.float32
    assert (c.head_dim, c.kv_heads, c.page_size) == (128, 2, 16)
    assert (c.desc.stride_page, c.desc.stride_head, c.desc.stride_row, c.desc.pages) == (2 * 16 * 128, 16 * 128, 128, 6)
    c = new(grid=E2M1, g=F16_ROW)
    assert c.k.shape == (6, 2, 16, 64) and c.head_dim == 128 and c.v_scales.dtype == torch.float16 and c.desc.stride_row == 64
    c = new(grid=None, g=None)
    assert c.k.dtype == torch.bfloat16 and c.k_scales is None and c.desc.stride_row == 256 and c.desc.type == L.FP4_BF16
    s = torch.ones(1)
    c = new(g=None, k_scale=s, v_scale=s.clone())
    assert c.gran.mode == L.FP4_SCALE_TENSOR and c.desc.k_scales == s.data_ptr()


def test_strides_of_caches():
    """Any order of pages, heads and slots; a dimension of one has no stride."""
    k, v = (torch.zeros(6, 16, 2, 64, dtype=torch.bfloat16).transpose(1, 2) for _ in range(2))
    d = F.KVCache(k, v).desc
    assert (d.stride_page, d.stride_head, d.stride_row) == (16 * 2 * 128, 128, 256)
    k, v = (torch.zeros(1, 16, 1, 64, dtype=torch.bfloat16).as_strided((1, 1, 16, 64), (7, 9, 64, 1)) for _ in range(2))
    d = F.KVCache(k, v).desc
    assert (d.stride_page, d.stride_head, d.stride_row) == (0, 0, 128)


def rows(dtype=torch.uint8, *shape):
    return torch.zeros(*(shape or (6, 2, 16, 128)), dtype=dtype)


S = torch.zeros(6, 2, 16)


@pytest.mark.parametrize("args", [
    (rows(torch.bfloat16), rows(torch.bfloat16), S, S), (rows(torch.float16), rows(torch.float16)), (rows(), rows()),
    (rows(torch.bfloat16), rows(torch.bfloat16), S, S, E4M3, ROW), (rows(), rows(torch.int8), S, S, E4M3, ROW),
    (rows(), rows(), S, S, E4M3), (rows(), rows(), None, S, E4M3, ROW), (rows(), rows(), S, None, E4M3, ROW),
    (rows(), rows(), S[:5], S, E4M3, ROW), (rows(), rows(), S, S.half(), E4M3, ROW), (rows(), rows(), S, S, E4M3, F16_ROW),
    (rows(), rows(), S, S, E4M3, ONE), (rows(), rows(), torch.zeros(1).half(), torch.zeros(1), E4M3, ONE),
    (rows(), rows(torch.uint8, 6, 2, 32, 128)[:, :, :16], S, S, E4M3, ROW), (rows(), rows(torch.uint8, 6, 2, 16, 64), S, S, E4M3, ROW),
    (rows().transpose(2, 3), rows().transpose(2, 3), S, S, E4M3, ROW), (rows()[0], rows()[0], S, S, E4M3, ROW),
    (rows(), rows(), S.transpose(0, 1).contiguous().transpose(0, 1), S, E4M3, ROW)])
def test_bad_caches(args):
    with pytest.raises(ValueError):
        F.KVCache(*args)


@pytest.mark.parametrize("kw", [dict(dim=80), dict(size=24), dict(size=8), dict(grid=F.grid_minifloat(2, 3)), dict(grid=F.grid_minifloat(1, 2))])
def test_unsupported_caches(host, kw):
    """What the library refuses comes back as its error, at the first call."""
    c = new(**kw)
    x = torch.zeros(3, 2, c.head_dim)
    with pytest.raises(F.FP4Error) as e:
        F.fp4_cache_write(x, x, c, ints(3, 2), ints(3))
    assert e.value.status == L.FP4_ERR_UNSUPPORTED


def test_overlapping_rows(host):
    """A cache of expanded pages, a write of expanded rows, a read into them."""
    c = F.KVCache(rows()[:1].expand(6, -1, -1, -1), rows()[:1].expand(6, -1, -1, -1), S, S, E4M3, ROW)
    x = torch.zeros(3, 2, 128)
    with pytest.raises(F.FP4Error):
        F.fp4_cache_write(x, x, c, ints(3, 2), ints(3))
    c, flat = new(), torch.zeros(1, 2, 128).expand(3, -1, -1)
    for k, v in ((flat, x), (x, flat)):
        with pytest.raises(F.FP4Error):
            F.fp4_cache_write(k, v, c, ints(3, 2), ints(3))
        with pytest.raises(F.FP4Error):
            F.fp4_cache_read(c, ints(3, 2), ints(3), k=k, v=v)
    with pytest.raises(F.FP4Error):
        F.fp4_cache_read(c, ints(3, 2), ints(3), k=x, v=x)
    with pytest.raises(F.FP4Error):
        F.fp4_attend(torch.zeros(3, 4, 128), c, ints(3, 2), ints(3), y=torch.zeros(1, 4, 128).expand(3, -1, -1))


X = torch.zeros(3, 2, 128)


@pytest.mark.parametrize("error,args", [
    (ValueError, (X, X.bfloat16(), None)), (TypeError, (X.half(), X.half(), None)), (ValueError, (X[:, :1], X, None)),
    (ValueError, (X, X[:2], None)), (ValueError, (X.view(3, 256), X, None)), (ValueError, (torch.zeros(3, 2, 96), X, None)),
    (ValueError, (torch.zeros(3, 128, 2).transpose(1, 2), X, None)), (ValueError, (torch.zeros(3, 4, 128)[:, ::2], X, None)),
    (ValueError, (X, X, ints(2))), (ValueError, (X, X, ints(3).long())), (ValueError, (X, X, ints(6)[::2]))])
def test_bad_rows(given, error, args):
    k, v, sequences = args
    c = new()
    with pytest.raises(error):
        F.fp4_cache_write(k, v, c, ints(3, 2), ints(3), sequences)
    with pytest.raises(error):
        F.fp4_cache_read(c, ints(3, 2), ints(3), sequences, k=k, v=v)
    for table, positions in ((ints(3, 2).long(), ints(3)), (ints(6), ints(3)), (ints(2, 3).t(), ints(3)), (ints(3, 2), ints(3).long()),
                             (ints(3, 2), ints(6)[::2])):
        with pytest.raises(ValueError):
            F.fp4_cache_write(X, X, c, table, positions)
    assert not given


@pytest.mark.parametrize("kw", [dict(q=torch.zeros(3, 4, 64)), dict(q=torch.zeros(3, 512)), dict(table=ints(2, 2)), dict(lengths=ints(2)),
                                dict(lengths=ints(3).long()), dict(y=torch.zeros(3, 2, 128)), dict(y=torch.zeros(2, 4, 128)),
                                dict(lse=torch.zeros(3, 2)), dict(lse=torch.zeros(3, 4).double()), dict(lse=torch.zeros(4, 3).t()),
                                dict(q=torch.zeros(3, 8, 128)[:, ::2]), dict(y=torch.zeros(3, 128, 4).transpose(1, 2)),
                                dict(workspace=torch.zeros(8, 1 << 20).t(), table=ints(3, 512)), dict(table=ints(3, 4)[:, ::2])])
def test_bad_attend(given, kw):
    a = dict(q=torch.zeros(3, 4, 128), table=ints(3, 2), lengths=ints(3), **{k: v for k, v in kw.items() if k not in ("q", "table", "lengths")})
    a.update(kw)
    with pytest.raises(ValueError):
        F.fp4_attend(a.pop("q"), new(), a.pop("table"), a.pop("lengths"), **a)
    assert not given


def test_unsupported_types():
    for kw in (dict(q=torch.zeros(3, 4, 128).half()), dict(q=torch.zeros(3, 4, 128), y_dtype=torch.float16)):
        with pytest.raises(TypeError):
            F.fp4_attend(kw.pop("q"), new(), ints(3, 2), ints(3), **kw)


def test_bad_numbers(host):
    q, c = torch.zeros(3, 4, 128), new()
    for kw in (dict(window=-1), dict(max_length=-1), dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=2.5e38), dict(scale=-2.5e38)):
        with pytest.raises(F.FP4Error) as e:
            F.fp4_attend(q, c, ints(3, 2), ints(3), **kw)
        assert e.value.status == L.FP4_ERR_INVALID_ARG
    with pytest.raises(F.FP4Error):
        F.fp4_attend(torch.zeros(3, 3, 128), c, ints(3, 2), ints(3))


def test_rows_as_given(given):
    """Columns of wider rows, a padded and a shared table, a single row of any stride."""
    c, wide = new(), torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    table, pos, seq = ints(5, 9)[:, :4], ints(3), ints(3)
    F.fp4_cache_write(wide[:, 4:6], wide[:, 6:], c, table, pos, seq)
    func, d = given.pop()
    assert func == "fp4_cache_write" and (d.sequences, d.max_pages, d.ld_table, d.tokens, d.ldk, d.ldv) == (5, 4, 9, 3, 1024, 1024)
    assert (d.k, d.v, d.dtype) == (wide.data_ptr() + 4 * 256, wide.data_ptr() + 6 * 256, L.FP4_BF16)
    assert (d.page_table, d.positions, d.sequence_of) == (table.data_ptr(), pos.data_ptr(), seq.data_ptr())
    k, v = F.fp4_cache_read(c, ints(1, 4).expand(3, -1), pos, dtype=torch.float32)
    func, d = given.pop()
    assert func == "fp4_cache_read" and d.ld_table == 0 and d.sequence_of is None and (d.k, d.v) == (k.data_ptr(), v.data_ptr())
    assert k.shape == v.shape == (3, 2, 128) and k.dtype == torch.float32 and d.dtype == L.FP4_F32
    one = torch.zeros(999).as_strided((1, 2, 128), (5, 128, 1))
    F.fp4_cache_write(one, one.clone(), c, ints(6).as_strided((1, 2), (3, 1)), ints(1))
    d = given.pop()[1]
    assert (d.ldk, d.ldv, d.ld_table) == (256, 256, 2)
    out = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    k, v = F.fp4_cache_read(c, table, pos, seq, v=out)
    assert v is out and k.dtype == out.dtype


def test_attend_as_given(given):
    c, wide = new(pages=4096), torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    y = F.fp4_attend(wide[:, :4], c, ints(3, 2), ints(3), window=7)
    _, d, ws, need = given.pop()
    assert (d.sequences, d.heads, d.ldq, d.ldy, d.max_pages, d.max_length, d.window) == (3, 4, 1024, 512, 2, 32, 7)
    assert y.shape == (3, 4, 128) and y.dtype == torch.bfloat16 and d.y_dtype == L.FP4_BF16 and d.scale == ctypes.c_float(128 ** -0.5).value
    assert ws is None and need == 0 and d.lse is None
    y = F.fp4_attend(wide[:, :4], c, ints(3, 4096), ints(3), scale=-0.5, max_length=9000, y_dtype=torch.float32, lse=torch.zeros(3, 4))
    _, d, ws, need = given.pop()
    assert (d.max_length, d.scale, d.y_dtype) == (9000, -0.5, L.FP4_F32) and y.dtype == torch.float32
    assert need == C._call("fp4_attend_workspace_size")(3, 4, 2, 128, 9000, 0) > 0 and ws
    # a workspace that is large enough is used, a smaller one is not
    room = torch.zeros(need, dtype=torch.uint8)
    F.fp4_attend(wide[:, :4], c, ints(3, 4096), ints(3), max_length=9000, workspace=room)
    assert given.pop()[2] == room.data_ptr()
    F.fp4_attend(wide[:, :4], c, ints(3, 4096), ints(3), max_length=9000, workspace=room[:-1])
    assert given.pop()[2] != room.data_ptr()
    F.fp4_attend(wide[:, :4], c, ints(3, 2), ints(3), max_length=10 ** 9)
    assert given.pop()[1].max_length == 32
