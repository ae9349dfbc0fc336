"""Binding of include/fp4_cache.h: a paged cache of keys and values as bf16 or as codes with scales,
rows written into it and read back, and the attention of one new token per sequence over it.

As the rest of the package, argument marshalling only: outputs are allocated here unless
the caller gives them, raw device pointers and the current HIP stream go to the C ABI, and
a non-OK status raises ``FP4Error``.  What the C side cannot see is checked here: devices,
element types, shapes and contiguity.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib as L
from .layer import _flat, _need, _raw_stream, _type

P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class fp4_kv_cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("pages", I64), ("stride_page", I64), ("stride_head", I64), ("stride_row", I64),
                ("kv_heads", I32), ("page_size", I32), ("head_dim", I32), ("type", I32), ("grid", L.fp4_grid),
                ("gran", L.fp4_gran), ("k_scales", P), ("v_scales", P)]


class fp4_cache_rows(ctypes.Structure):
    _fields_ = [("page_table", P), ("sequences", I64), ("max_pages", I64), ("ld_table", I64), ("positions", P),
                ("sequence_of", P)]


class fp4_attend_desc(ctypes.Structure):
    _fields_ = [("sequences", I64), ("heads", I32), ("q_dtype", I32), ("q", P), ("ldq", I64), ("page_table", P),
                ("max_pages", I64), ("ld_table", I64), ("lengths", P), ("max_length", I64), ("window", I64), ("scale", F32),
                ("y_dtype", I32), ("y", P), ("ldy", I64), ("lse", P)]


_CACHE, _ROWS, _ATTEND = (ctypes.POINTER(t) for t in (fp4_kv_cache, fp4_cache_rows, fp4_attend_desc))
SIGNATURES = {
    "fp4_cache_write": (I32, [_CACHE, _ROWS, I64, P, I64, P, I64, I32, P]),
    "fp4_cache_read": (I32, [_CACHE, _ROWS, I64, P, I64, P, I64, I32, P]),
    "fp4_attend_workspace_size": (ctypes.c_size_t, [I64, I32, I32, I32, I64, I64]),
    "fp4_attend": (I32, [_CACHE, _ATTEND, P, ctypes.c_size_t, P]),
}

_entry = {}


def _call(name):
    f = _entry.get(name)
    if f is None:
        lib = L.lib()
        for n, (res, args) in SIGNATURES.items():
            g = getattr(lib, n)
            g.restype, g.argtypes = res, args
            _entry[n] = g
        f = _entry[name]
    return f


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(dev, func, *args):
    """A call on a device's current stream, with that device current."""
    f = _call(func)
    if dev.index == _current_device() and _raw_stream is not None:
        status = f(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = f(*args, torch.cuda.current_stream(dev).cuda_stream)
    if status:
        L.check(status, func)


class KVCache:
    """A paged cache that the caller's tensors hold.

    k, v: [pages, kv_heads, page_size, head_dim] bf16, or uint8 codes of `grid` (E2M1 packed: head_dim / 2 bytes
    a row), in any order of strides that keeps a row contiguous (the same for both).  Codes have scales: with
    g = gran("row") one a row, f32 or f16 [pages, kv_heads, page_size] contiguous; with g = gran("tensor") one
    f32 value each, given.  The object keeps the tensors; make it once and use it for every call."""
    __slots__ = ("k", "v", "k_scales", "v_scales", "grid", "gran", "head_dim", "kv_heads", "page_size", "device", "desc")

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor | None = None,
                 v_scales: torch.Tensor | None = None, grid: L.fp4_grid | None = None, g: L.fp4_gran | None = None):
        _need(k.dim() == 4, "k and v must be [pages, kv_heads, page_size, row]")
        kind = torch.bfloat16 if grid is None else torch.uint8
        _need(k.dtype == kind and v.dtype == kind, f"the rows of this cache must be {kind}")
        _need(v.shape == k.shape and v.stride() == k.stride() and v.device == k.device, "k and v must have one shape, layout and device")
        _need(k.stride(3) == 1, "a row must be contiguous")
        (pages, heads, size, width), dev = k.shape, k.device
        if grid is None:
            _need(k_scales is None and v_scales is None, "a bf16 cache has no scales")
            g = L.fp4_gran()
        else:
            _need(g is not None, "a grid needs a granularity")
            count = pages * heads * size if g.mode == L.FP4_SCALE_ROW else 1
            dtype = torch.float16 if g.scale_dtype == L.FP4_F16 and g.mode == L.FP4_SCALE_ROW else torch.float32
            for name, s in (("k_scales", k_scales), ("v_scales", v_scales)):
                _need(s is not None, f"a cache of codes needs {name}")
                _flat(s, name, count, dtype, dev)
        # a dimension of one may have any stride
        strides = [st * k.element_size() if n > 1 else 0 for n, st in zip(k.shape, k.stride())]
        self.k, self.v, self.k_scales, self.v_scales, self.grid, self.gran = k, v, k_scales, v_scales, grid, g
        self.head_dim = width * (2 if grid is not None and (grid.e, grid.m) == (2, 1) else 1)
        self.kv_heads, self.page_size, self.device = heads, size, dev
        self.desc = fp4_kv_cache(
            k.data_ptr(), v.data_ptr(), pages, *strides[:3], heads, size, self.head_dim, L.FP4_BF16 if grid is None else L.FP4_PACKED,
            grid if grid is not None else L.fp4_grid(), g, k_scales.data_ptr() if k_scales is not None else None,
            v_scales.data_ptr() if v_scales is not None else None)


def kv_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, grid: L.fp4_grid | None = None,
             g: L.fp4_gran | None = None, k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
             device="cuda") -> KVCache:
    """A new cache of zeros: bf16 without a grid, else codes with a scale per row (g = gran("row"), the default) or
    with the given k_scale and v_scale (f32, one value each; g = gran("tensor"))."""
    if grid is None:
        shape, kind = (pages, kv_heads, page_size, head_dim), torch.bfloat16
    else:
        _need(not (head_dim % 2 and (grid.e, grid.m) == (2, 1)), "head_dim must be even")
        shape, kind = (pages, kv_heads, page_size, head_dim // (2 if (grid.e, grid.m) == (2, 1) else 1)), torch.uint8
        if g is None:
            g = L.fp4_gran(L.FP4_SCALE_TENSOR if k_scale is not None else L.FP4_SCALE_ROW, 0, L.FP4_F32, 0)
        if g.mode == L.FP4_SCALE_ROW:
            _need(k_scale is None and v_scale is None, "k_scale and v_scale need gran('tensor')")
            k_scale, v_scale = (torch.zeros(shape[:3], dtype=torch.float16 if g.scale_dtype == L.FP4_F16 else torch.float32, device=device)
                                for _ in range(2))
    return KVCache(torch.zeros(shape, dtype=kind, device=device), torch.zeros(shape, dtype=kind, device=device), k_scale, v_scale, grid, g)


# The checks below run on every call, beside kernels of a few microseconds.
def _heads(t, name, rows, heads, dim, dev):
    """Leading dimension of rows of heads: [rows, heads, dim], the heads of a row side by side."""
    if t.shape != (rows, heads, dim) or t.device != dev:
        raise ValueError(f"{name} must be [{rows}, {heads}, {dim}] on {dev}, not {list(t.shape)} on {t.device}")
    ld, head, step = t.stride()
    if step != 1 or (head != dim and heads > 1):
        raise ValueError(f"the heads of {name} must lie side by side")
    return ld if rows > 1 or ld > heads * dim else heads * dim


def _table(t, dev):
    """Sizes of a page table: rows, columns, leading dimension."""
    if t.dim() != 2 or t.dtype != torch.int32 or t.device != dev or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"page_table must be int32 [sequences, pages] on {dev}, row-major")
    rows, cols = t.shape
    return rows, cols, (t.stride(0) if rows > 1 or t.stride(0) > cols else cols)


def _rows(cache, page_table, positions, sequences):
    dev = cache.device
    if positions.dim() != 1:
        raise ValueError("positions must be one list")
    n = positions.shape[0]
    rows, cols, ld = _table(page_table, dev)
    return n, fp4_cache_rows(page_table.data_ptr(), rows, cols, ld, _flat(positions, "positions", n, torch.int32, dev),
                             _flat(sequences, "sequences", n, torch.int32, dev))


def fp4_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor, positions: torch.Tensor,
                    sequences: torch.Tensor | None = None) -> None:
    """Keys and values of tokens (k, v [tokens, kv_heads, head_dim], f32 / bf16) into the cache.

    Token i becomes position positions[i] (int32) of sequence sequences[i] (int32; i itself without them), in page
    page_table[sequence, position // page_size] (int32 [sequences, pages]).  Tokens whose position is negative or past
    the table, or whose page is not in the cache, are skipped (padding).  No two tokens may have one place."""
    n, rows = _rows(cache, page_table, positions, sequences)
    heads, dim, dev = cache.kv_heads, cache.head_dim, cache.device
    if k.dtype != v.dtype:
        raise ValueError("k and v must have one dtype")
    _launch(dev, "fp4_cache_write", cache.desc, rows, n, k.data_ptr(), _heads(k, "k", n, heads, dim, dev), v.data_ptr(),
            _heads(v, "v", n, heads, dim, dev), _type(k, "k"))


def fp4_cache_read(cache: KVCache, page_table: torch.Tensor, positions: torch.Tensor, sequences: torch.Tensor | None = None,
                   dtype: torch.dtype = torch.bfloat16, k: torch.Tensor | None = None, v: torch.Tensor | None = None):
    """The keys and values that the cache holds for tokens given as in fp4_cache_write, as (k, v)
    [tokens, kv_heads, head_dim]; zeros for tokens without a place."""
    n, rows = _rows(cache, page_table, positions, sequences)
    heads, dim, dev = cache.kv_heads, cache.head_dim, cache.device
    if k is None:
        k = torch.empty((n, heads, dim), dtype=dtype if v is None else v.dtype, device=dev)
    if v is None:
        v = torch.empty((n, heads, dim), dtype=k.dtype, device=dev)
    if k.dtype != v.dtype:
        raise ValueError("k and v must have one dtype")
    _launch(dev, "fp4_cache_read", cache.desc, rows, n, k.data_ptr(), _heads(k, "k", n, heads, dim, dev), v.data_ptr(),
            _heads(v, "v", n, heads, dim, dev), _type(k, "k"))
    return k, v


def fp4_attend(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, lengths: torch.Tensor, scale: float | None = None,
               window: int = 0, max_length: int | None = None, y: torch.Tensor | None = None,
               y_dtype: torch.dtype | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of one new token per sequence over its positions in the cache.

    q: [sequences, heads, head_dim] f32 / bf16, heads a multiple of the cache's kv_heads (groups of query heads
    share one); lengths: int32 [sequences], the new token's own position counted (write it first); scale: factor of
    the products (head_dim ** -0.5); window: the last so many positions only; max_length: no length is larger (the page
    table's, unless given: a smaller one saves launching parts that have no positions).  Returns y of q's shape (q's dtype
    unless y or y_dtype is given); a sequence that sees nothing has zeros.  lse (f32 [sequences, heads]) takes the logarithms of
    the sums of exponentials.  A drafted token is a sequence of its own with the same row of the table."""
    _need(q.dim() == 3, "q must be [sequences, heads, head_dim]")
    (n, heads, dim), dev = q.shape, cache.device
    _need(dim == cache.head_dim, "q must have the cache's head_dim")
    if y is None:
        y = torch.empty((n, heads, dim), dtype=y_dtype or q.dtype, device=dev)
    rows, cols, ld = _table(page_table, dev)
    if rows != n:
        raise ValueError(f"page_table must have a row for each of {n} sequences")
    most = cols * cache.page_size
    if max_length is not None and max_length < most:
        most = max_length
    need = _call("fp4_attend_workspace_size")(n, heads, cache.kv_heads, dim, most, window)
    if need:
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous memory on {dev}")
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    d = fp4_attend_desc(
        n, heads, _type(q, "q"), q.data_ptr(), _heads(q, "q", n, heads, dim, dev), page_table.data_ptr(), cols, ld,
        _flat(lengths, "lengths", n, torch.int32, dev), most, window, dim ** -0.5 if scale is None else scale, _type(y, "y"),
        y.data_ptr(), _heads(y, "y", n, heads, dim, dev), _flat(lse, "lse", n * heads, torch.float32, dev))
    _launch(dev, "fp4_attend", cache.desc, d, workspace.data_ptr() if need else None, need)
    return y
