"""Binding of include/fp4_cache.h: a paged cache of keys and values as bf16 or as codes with scales,
rows written into it and read back, and the attention of one new token per sequence over it.

As the rest of the package, argument marshalling only: outputs are allocated here unless
the caller gives them, raw device pointers and the current HIP stream go to the C ABI, and
a non-OK status raises ``FP4Error``.  What the C side cannot see is checked here: devices,
element types, shapes and contiguity.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _lib as L
from .layer import _TYPES, _flat, _need, _raw_stream

P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class fp4_kv_cache(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("pages", I64), ("stride_page", I64), ("stride_head", I64), ("stride_row", I64),
                ("kv_heads", I32), ("page_size", I32), ("head_dim", I32), ("type", I32), ("grid", L.fp4_grid),
                ("gran", L.fp4_gran), ("k_scales", P), ("v_scales", P)]


class fp4_cache_rows_desc(ctypes.Structure):
    _fields_ = [("page_table", P), ("sequences", I64), ("max_pages", I64), ("ld_table", I64), ("tokens", I64), ("positions", P),
                ("sequence_of", P), ("k", P), ("ldk", I64), ("v", P), ("ldv", I64), ("dtype", I32), ("reserved", I32)]


class fp4_attend_desc(ctypes.Structure):
    _fields_ = [("sequences", I64), ("heads", I32), ("q_dtype", I32), ("q", P), ("ldq", I64), ("page_table", P),
                ("max_pages", I64), ("ld_table", I64), ("lengths", P), ("max_length", I64), ("window", I64), ("scale", F32),
                ("y_dtype", I32), ("y", P), ("ldy", I64), ("lse", P)]


# descriptors of a call go as bytes (see _pack), the cache's as it is kept
_CACHE, _DESC = ctypes.POINTER(fp4_kv_cache), ctypes.c_char_p
SIGNATURES = {
    "fp4_cache_write": (I32, [_CACHE, _DESC, P]),
    "fp4_cache_read": (I32, [_CACHE, _DESC, P]),
    "fp4_attend_workspace_size": (ctypes.c_size_t, [I64, I32, I32, I32, I64, I64]),
    "fp4_attend": (I32, [_CACHE, _DESC, P, ctypes.c_size_t, P]),
}


def _pack(struct_type):
    """A function that packs the fields of a descriptor (pointers as numbers, 0 for none) into its bytes: a call on a
    few tokens takes as long as its marshalling, and a ctypes structure costs four times this."""
    codes = {P: "P", I64: "q", I32: "i", F32: "f"}
    s = struct.Struct("@" + "".join(codes[f[1]] for f in struct_type._fields_))
    assert s.size == ctypes.sizeof(struct_type)
    return s.pack


_rows_desc, _attend_desc = _pack(fp4_cache_rows_desc), _pack(fp4_attend_desc)

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


def _launch(cache, func, *args):
    """A call on a cache, on its device's current stream and with that device current."""
    f = _entry.get(func) or _call(func)
    if _raw_stream is not None and cache.index == _current_device():
        status = f(cache.desc, *args, _raw_stream(cache.index))
    else:
        with torch.cuda.device(cache.device):
            status = f(cache.desc, *args, torch.cuda.current_stream(cache.device).cuda_stream)
    if status:
        L.check(status, func)


@functools.lru_cache(4096)
def _workspace_size(*sizes):
    return _call("fp4_attend_workspace_size")(*sizes)


class KVCache:
    """A paged cache that the caller's tensors hold.

    k, v: [pages, kv_heads, page_size, head_dim] bf16, or uint8 codes of `grid` (E2M1 packed: head_dim / 2 bytes
    a row), in any order of strides that keeps a row contiguous (the same for both).  Codes have scales: with
    g = gran("row") one a row, f32 or f16 [pages, kv_heads, page_size] contiguous; with g = gran("tensor") one
    f32 value each, given.  The object keeps the tensors; make it once and use it for every call.  Its descriptor holds
    their addresses, so its fields are set once: for other tensors make a new object."""
    __slots__ = ("k", "v", "k_scales", "v_scales", "grid", "gran", "head_dim", "kv_heads", "page_size", "device", "index", "desc")

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
        self.kv_heads, self.page_size, self.device, self.index = heads, size, dev, k.get_device()
        self.desc = fp4_kv_cache(
            k.data_ptr(), v.data_ptr(), pages, *strides[:3], heads, size, self.head_dim, L.FP4_BF16 if grid is None else L.FP4_PACKED,
            grid if grid is not None else L.fp4_grid(), g, k_scales.data_ptr() if k_scales is not None else None,
            v_scales.data_ptr() if v_scales is not None else None)

    def __setattr__(self, name, value):
        if hasattr(self, name):
            raise AttributeError(f"{name} of a cache cannot be replaced: make a new KVCache")
        super().__setattr__(name, value)

    def __delattr__(self, name):
        raise AttributeError(f"{name} of a cache cannot be deleted: make a new KVCache")


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


# The checks below run on every call, beside kernels of a few microseconds: one condition each, the message
# made only when it fails.  (Devices are compared by their number, -1 for none.)
def _heads(t, name, shape, cache):
    """Leading dimension of rows of heads [rows, heads, dim], the heads of a row side by side."""
    if t.shape != shape or t.get_device() != cache.index:
        raise ValueError(f"{name} must be {list(shape)} on {cache.device}, not {list(t.shape)} on {t.device}")
    ld, head, step = t.stride()
    rows, heads, dim = shape
    if step != 1 or (head != dim and heads > 1):
        raise ValueError(f"the heads of {name} must lie side by side")
    return ld if rows > 1 else heads * dim  # the stride of a single row means nothing


def _table(t, cache):
    """Sizes of a page table: rows, columns, leading dimension."""
    shape = t.shape
    if len(shape) != 2 or t.dtype != torch.int32 or t.get_device() != cache.index:
        raise ValueError(f"page_table must be int32 [sequences, pages] on {cache.device}")
    rows, cols = shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError("page_table must be row-major")
    return rows, cols, (ld if rows > 1 else cols)


def _list(t, name, count, dtype, cache):
    """Pointer of a contiguous tensor of `count` values (None: 0)."""
    if t is None:
        return 0
    if t.numel() != count or t.dtype != dtype or t.get_device() != cache.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} values on {cache.device}")
    return t.data_ptr()


def _float(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _rows_call(func, k, v, cache, page_table, positions, sequences):
    n = positions.numel()
    shape = (n, cache.kv_heads, cache.head_dim)
    kind = _float(k, "k")
    if v.dtype != k.dtype:
        raise ValueError("k and v must have one dtype")
    _launch(cache, func, _rows_desc(
        page_table.data_ptr(), *_table(page_table, cache), n, _list(positions, "positions", n, torch.int32, cache),
        _list(sequences, "sequences", n, torch.int32, cache), k.data_ptr(), _heads(k, "k", shape, cache), v.data_ptr(),
        _heads(v, "v", shape, cache), kind, 0))


def fp4_cache_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor, positions: torch.Tensor,
                    sequences: torch.Tensor | None = None) -> None:
    """Keys and values of tokens (k, v [tokens, kv_heads, head_dim], f32 / bf16) into the cache.

    Token i becomes position positions[i] (int32) of sequence sequences[i] (int32; i itself without them), in page
    page_table[sequence, position // page_size] (int32 [sequences, pages]).  Tokens whose position is negative or past
    the table, or whose page is not in the cache, are skipped (padding).  No two tokens may have one place."""
    _rows_call("fp4_cache_write", k, v, cache, page_table, positions, sequences)


def fp4_cache_read(cache: KVCache, page_table: torch.Tensor, positions: torch.Tensor, sequences: torch.Tensor | None = None,
                   dtype: torch.dtype = torch.bfloat16, k: torch.Tensor | None = None, v: torch.Tensor | None = None):
    """The keys and values that the cache holds for tokens given as in fp4_cache_write, as (k, v)
    [tokens, kv_heads, head_dim]; zeros for tokens without a place."""
    shape = (positions.numel(), cache.kv_heads, cache.head_dim)
    if k is None:
        k = torch.empty(shape, dtype=dtype if v is None else v.dtype, device=cache.device)
    if v is None:
        v = torch.empty(shape, dtype=k.dtype, device=cache.device)
    _rows_call("fp4_cache_read", k, v, cache, page_table, positions, sequences)
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
    the sums of exponentials.  workspace: device memory that is used if it is large enough (else the call makes its own); calls
    that may overlap in time need one each.  A drafted token is a sequence of its own with the same row of the table.

    Scores and sums are binary32: |scale| log2(e) times the sum of |q k| (codes of k, before their row's scale) and 2^8 times the sum of |v|
    over a sequence's positions must stay finite, and |z| log2(e) below 1.5e38 (include/fp4_cache.h)."""
    shape, dim = q.shape, cache.head_dim
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError(f"q must be [sequences, heads, {dim}]")
    n, heads, _ = shape
    if y is None:
        y = torch.empty(shape, dtype=y_dtype or q.dtype, device=cache.device)
    rows, cols, ld = _table(page_table, cache)
    if rows != n:
        raise ValueError(f"page_table must have a row for each of {n} sequences")
    most = cols * cache.page_size
    if max_length is not None and max_length < most:
        most = max_length
    need, at = _workspace_size(n, heads, cache.kv_heads, dim, most, window), None
    if need:
        if workspace is not None and (workspace.get_device() != cache.index or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous memory on {cache.device}")
        if workspace is None or workspace.numel() * workspace.element_size() < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=cache.device)
        at = workspace.data_ptr()
    _launch(cache, "fp4_attend", _attend_desc(
        n, heads, _float(q, "q"), q.data_ptr(), _heads(q, "q", shape, cache), page_table.data_ptr(), cols, ld,
        _list(lengths, "lengths", n, torch.int32, cache), most, window, dim ** -0.5 if scale is None else scale, _float(y, "y"),
        y.data_ptr(), _heads(y, "y", shape, cache), _list(lse, "lse", n * heads, torch.float32, cache)), at, need)
    return y
