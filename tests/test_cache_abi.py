"""include/fp4_cache.h without a GPU: the library exports what the header declares with the
binding's layouts, and bad arguments come back from the host with their status before
anything is launched."""
import ctypes
import os
import re
import subprocess

import pytest

from bit_floating_point_amd import _lib as L
from bit_floating_point_amd import cache as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp4_cache.h")
FAKE, OTHER, ODD = 0x10000, 0x20000, 0x10008  # never dereferenced: every call below is refused first
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (L.FP4_OK, L.FP4_ERR_INVALID_ARG, L.FP4_ERR_UNSUPPORTED, L.FP4_ERR_ALIGNMENT,
                                                  L.FP4_ERR_WORKSPACE)


def grid(e=4, m=3, kind=0):
    g = L.fp4_grid()
    g.kind, g.e, g.m = kind, e, m
    return g


def gran(mode=1, group=0, sd=0, reserved=0):
    return L.fp4_gran(mode, group, sd, reserved)


def cache(**kw):
    """Four pages of 16 slots, two heads of 128, E4M3 with f32 scales."""
    c = C.fp4_kv_cache(k=FAKE, v=OTHER, pages=4, stride_page=4096, stride_head=2048, stride_row=128, kv_heads=2, page_size=16,
                       head_dim=128, type=L.FP4_PACKED, grid=grid(), gran=gran(), k_scales=FAKE, v_scales=FAKE)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def call(name, c, d, *more):
    """A descriptor as the library's C callers give it."""
    return C._call(name)(c, None if d is None else bytes(d), *more)


def rows(**kw):
    r = C.fp4_cache_rows_desc(page_table=FAKE, sequences=3, max_pages=2, ld_table=2, tokens=5, positions=FAKE, sequence_of=None, k=FAKE,
                              ldk=256, v=OTHER, ldv=256, dtype=L.FP4_BF16)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def move(name, c=None, **kw):
    return call(name, c or cache(), rows(**kw), None)


def attend(c=None, ws=FAKE, ws_bytes=1 << 30, **kw):
    d = C.fp4_attend_desc(sequences=3, heads=4, q_dtype=L.FP4_BF16, q=FAKE, ldq=512, page_table=FAKE, max_pages=2, ld_table=2,
                          lengths=FAKE, max_length=32, window=0, scale=1.0, y_dtype=L.FP4_BF16, y=OTHER, ldy=512, lse=None)
    for k, v in kw.items():
        setattr(d, k, v)
    return call("fp4_attend", c or cache(), d, ws, ws_bytes, None)


def test_exports_and_signatures():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(fp4_[a-z_0-9]+)\s*\(", text))
    assert names == set(C.SIGNATURES)
    lib = L.load()
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("struct", [C.fp4_kv_cache, C.fp4_cache_rows_desc, C.fp4_attend_desc])
def test_struct_layouts(struct, tmp_path):
    fields = [f[0] for f in struct._fields_]
    src = tmp_path / "s.c"
    src.write_text('#include "fp4_cache.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(void){printf("%zu",sizeof('
                   + struct.__name__ + "));" + "".join(f'printf(" %zu", offsetof({struct.__name__}, {f}));' for f in fields)
                   + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = [int(v) for v in subprocess.check_output([str(exe)]).split()]
    assert got == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


BF16 = dict(type=L.FP4_BF16, k_scales=None, v_scales=None, stride_row=256, stride_head=4096, stride_page=8192)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(v=FAKE)), (INVALID, dict(pages=0)), (INVALID, dict(pages=-1)),
    (INVALID, dict(pages=1 << 31)), (INVALID, dict(kv_heads=0)), (INVALID, dict(kv_heads=65536)), (INVALID, dict(type=L.FP4_F32)),
    (INVALID, dict(type=9)), (INVALID, dict(k_scales=None)), (INVALID, dict(v_scales=None)), (INVALID, dict(gran=gran(9))),
    (INVALID, dict(gran=gran(1, 0, 5))), (INVALID, dict(gran=gran(reserved=1))), (INVALID, dict(grid=grid(kind=7))),
    (INVALID, dict(BF16, k_scales=FAKE)), (INVALID, dict(stride_row=112)), (INVALID, dict(stride_row=0)), (INVALID, dict(stride_row=-128)),
    (INVALID, dict(stride_head=2032)), (INVALID, dict(stride_page=0)), (INVALID, dict(stride_page=4080)),
    (INVALID, dict(BF16, stride_row=128)), (INVALID, dict(stride_page=-4096)), (INVALID, dict(stride_head=8192)),
    (UNSUPPORTED, dict(page_size=8)), (UNSUPPORTED, dict(page_size=24)), (UNSUPPORTED, dict(page_size=0)), (UNSUPPORTED, dict(page_size=1 << 17)),
    (UNSUPPORTED, dict(head_dim=80)), (UNSUPPORTED, dict(head_dim=512)), (UNSUPPORTED, dict(head_dim=0)), (UNSUPPORTED, dict(grid=grid(1, 2))),
    (UNSUPPORTED, dict(grid=grid(2, 3))), (UNSUPPORTED, dict(grid=grid(0, 0, 2))), (UNSUPPORTED, dict(gran=gran(2, 64))),
    (UNSUPPORTED, dict(gran=gran(0, 0, L.FP4_F16))), (UNSUPPORTED, dict(stride_row=1 << 28, stride_head=1 << 32, stride_page=1 << 33)),
    (UNSUPPORTED, dict(stride_page=1 << 60)), (UNSUPPORTED, dict(stride_head=1 << 61, stride_page=2048)),
    (ALIGNMENT, dict(k=ODD)), (ALIGNMENT, dict(v=ODD)), (ALIGNMENT, dict(k_scales=ODD)), (ALIGNMENT, dict(stride_row=136, stride_head=4096, stride_page=8192)),
    (ALIGNMENT, dict(stride_head=2056, stride_page=8192)), (ALIGNMENT, dict(stride_page=4104))])
def test_bad_caches(status, kw):
    """The same rule in every call; tokens and sequences are there, so nothing returns early."""
    for name in ("fp4_cache_write", "fp4_cache_read"):
        assert move(name, cache(**kw)) == status, L.lib().fp4_last_error()
    assert attend(cache(**kw)) == status, L.lib().fp4_last_error()


@pytest.mark.parametrize("kw", [dict(), dict(BF16), dict(stride_head=128, stride_row=256), dict(stride_page=128, stride_row=512, stride_head=8192),
                                dict(pages=1, stride_page=0), dict(kv_heads=1, stride_head=0), dict(grid=grid(2, 1), stride_row=64),
                                dict(grid=grid(5, 2), gran=gran(0)), dict(gran=gran(1, 0, L.FP4_F16)), dict(stride_page=1 << 40)])
def test_good_caches(kw):
    """Any order of strides, and gaps; no tokens, so nothing is launched."""
    for name in ("fp4_cache_write", "fp4_cache_read"):
        assert move(name, cache(**kw), tokens=0) == OK, L.lib().fp4_last_error()


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(tokens=-1)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(ldk=255)), (INVALID, dict(ldv=128)),
    (INVALID, dict(dtype=L.FP4_F16)), (INVALID, dict(reserved=1)), (INVALID, dict(page_table=None)), (INVALID, dict(positions=None)),
    (INVALID, dict(sequences=-1)), (INVALID, dict(sequences=1 << 31)), (INVALID, dict(max_pages=-1)),
    (INVALID, dict(ld_table=1)), (UNSUPPORTED, dict(max_pages=(1 << 26) + 1, ld_table=1 << 27)),
    (UNSUPPORTED, dict(ld_table=1 << 60)), (UNSUPPORTED, dict(tokens=1 << 40, ldk=1 << 40)),
    (ALIGNMENT, dict(k=ODD)), (ALIGNMENT, dict(v=ODD)), (ALIGNMENT, dict(ldk=260)), (ALIGNMENT, dict(page_table=0x10002)),
    (ALIGNMENT, dict(positions=0x10002)), (ALIGNMENT, dict(sequence_of=0x10001))])
def test_bad_rows(status, kw):
    for name in ("fp4_cache_write", "fp4_cache_read"):
        assert move(name, **kw) == status, L.lib().fp4_last_error()


def test_rows_that_nobody_has():
    """No tokens: nothing to do.  No sequences or no pages: nothing to write."""
    for name in ("fp4_cache_write", "fp4_cache_read"):
        assert move(name, tokens=0, k=None, v=None, positions=None) == OK
        assert call(name, None, rows(), None) == INVALID
        assert call(name, cache(), None, None) == INVALID
    assert move("fp4_cache_write", sequences=0, page_table=None) == OK
    assert move("fp4_cache_write", max_pages=0, page_table=None) == OK
    assert move("fp4_cache_read", v=FAKE) == INVALID


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(y=None)), (INVALID, dict(lengths=None)), (INVALID, dict(page_table=None)), (INVALID, dict(heads=3)),
    (INVALID, dict(heads=0)), (INVALID, dict(heads=-2)), (INVALID, dict(sequences=-1)), (INVALID, dict(q_dtype=L.FP4_F16)),
    (INVALID, dict(y_dtype=7)), (INVALID, dict(ldq=511)), (INVALID, dict(ldy=256)), (INVALID, dict(max_length=-1)), (INVALID, dict(window=-1)),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(scale=float("inf"))), (INVALID, dict(ld_table=1)), (INVALID, dict(max_pages=-1)),
    (UNSUPPORTED, dict(heads=65538)), (UNSUPPORTED, dict(max_pages=1 << 27, ld_table=1 << 27)), (UNSUPPORTED, dict(sequences=1 << 30, ldq=1 << 31)),
    (ALIGNMENT, dict(q=ODD)), (ALIGNMENT, dict(y=ODD)), (ALIGNMENT, dict(ldq=516)), (ALIGNMENT, dict(ldy=516)), (ALIGNMENT, dict(lengths=0x10002)),
    (ALIGNMENT, dict(lse=0x10001)), (ALIGNMENT, dict(ws=ODD)), (ALIGNMENT, dict(page_table=0x10001)),
    (WORKSPACE, dict(ws=None, max_pages=1 << 10, ld_table=1 << 10, max_length=1 << 14)),
    (WORKSPACE, dict(ws_bytes=1024, max_pages=1 << 10, ld_table=1 << 10, max_length=1 << 14))])
def test_bad_attend(status, kw):
    assert attend(**kw) == status, L.lib().fp4_last_error()


def test_attend_of_no_sequences():
    assert attend(sequences=0, q=None, y=None, lengths=None, page_table=None) == OK
    assert call("fp4_attend", None, C.fp4_attend_desc(), None, 0, None) == INVALID
    assert call("fp4_attend", cache(), None, None, 0, None) == INVALID


def test_workspace_size():
    """None for short sequences and large batches; never less for a longer bound, so that the workspace of a page table's
    whole length serves every max_length; 0 for sizes that fp4_attend refuses."""
    size = C._call("fp4_attend_workspace_size")
    assert size(1, 32, 32, 128, 1, 0) == 0 and size(4096, 40, 40, 128, 1 << 20, 0) == 0
    for n, heads, kv in ((1, 8, 8), (3, 40, 8), (17, 64, 1), (300, 5, 5)):
        last = 0
        for length in list(range(1, 3000, 13)) + [1 << e for e in range(12, 34)]:
            now = size(n, heads, kv, 128, length, 0)
            assert now >= last and now % (4 * n * heads) == 0
            last = now
        assert size(n, heads, kv, 128, 1 << 33, 0) == size(n, heads, kv, 128, 1 << 30, 0)
    for bad in ((0, 8, 8, 128, 9, 0), (-1, 8, 8, 128, 9, 0), (1, 9, 8, 128, 9, 0), (1, 0, 8, 128, 9, 0), (1, 8, 0, 128, 9, 0),
                (1, 8, 8, 0, 9, 0), (1, 8, 8, 128, -1, 0), (1, 8, 8, 128, 9, -1), (1 << 40, 8, 8, 128, 9, 0)):
        assert size(*bad) == 0
