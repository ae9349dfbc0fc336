"""Scales per row of keys and of values are two arrays: a write into a cache where they share memory would leave each row's keys
or values with the other's scale, so it is refused, on the host.  One given scale may serve both, and what only reads may
share.  No GPU: nothing is launched."""
import pytest
import torch

import bit_floating_point_amd as F
from bit_floating_point_amd import _lib as L
from bit_floating_point_amd import cache as C
from test_cache_abi import FAKE, cache, call, gran, rows

APART = 0x40000  # rows of k and v end below
HALF = gran(1, 0, L.FP4_F16)
BYTES = 4 * 2 * 16 * 4  # f32 scales of the cache of test_cache_abi


def write(status, message=b"", **kw):
    got = call("fp4_cache_write", cache(**kw), rows(), None)
    assert got == status and message in L.lib().fp4_last_error(), L.lib().fp4_last_error()


@pytest.mark.parametrize("off", [0, 16, BYTES - 16, -16, 16 - BYTES])
def test_shared_row_scales(off):
    write(L.FP4_ERR_INVALID_ARG, b"k_scales and v_scales", k_scales=APART, v_scales=APART + off)


@pytest.mark.parametrize("off", [0, BYTES // 2 - 16, 16 - BYTES // 2])
def test_shared_f16_scales(off):
    write(L.FP4_ERR_INVALID_ARG, b"k_scales and v_scales", k_scales=APART, v_scales=APART + off, gran=HALF)


def test_the_largest_cache():
    """Counts whose bytes pass 32 bits: pages of the largest size, v_scales a page short of the end of k_scales."""
    big = dict(pages=1 << 20, page_size=1 << 16, kv_heads=1, stride_head=0, stride_page=128 << 16)
    write(L.FP4_ERR_INVALID_ARG, b"k_scales and v_scales", k_scales=1 << 50, v_scales=(1 << 50) + (1 << 38) - (1 << 18), **big)


def test_what_else_is_wrong_comes_first():
    """Nothing to write is nothing wrong; a bad pointer keeps its own message."""
    assert call("fp4_cache_write", cache(), rows(tokens=0), None) == L.FP4_OK
    assert call("fp4_cache_write", cache(), rows(sequences=0, page_table=None), None) == L.FP4_OK
    write(L.FP4_ERR_INVALID_ARG, b"needs k_scales", k_scales=None)
    write(L.FP4_ERR_ALIGNMENT, b"16 bytes", k_scales=FAKE + 8, v_scales=FAKE + 8)


def test_binding():
    """The package's call, to the library's host checks."""
    s, k, v = torch.zeros(6, 2, 16), torch.zeros(6, 2, 16, 128, dtype=torch.uint8), torch.zeros(6, 2, 16, 128, dtype=torch.uint8)
    c = F.KVCache(k, v, s, s, F.grid_minifloat(4, 3), F.gran("row"))
    x, ints = torch.zeros(3, 2, 128), torch.zeros(3, 2, dtype=torch.int32)
    d = C._rows_desc(ints.data_ptr(), 3, 2, 2, 3, ints.data_ptr(), 0, x.data_ptr(), 256, x.data_ptr(), 256, L.FP4_F32, 0)
    with pytest.raises(F.FP4Error, match="k_scales and v_scales"):
        L.check(C._call("fp4_cache_write")(c.desc, d, None), "fp4_cache_write")
