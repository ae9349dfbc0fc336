"""Binding of include/fp4_layer.h: the norm and SwiGLU with 8-bit outputs, the product of
8-bit operands with block scales, the routing of tokens to experts and the experts'
products.

As the rest of the package, argument marshalling only: outputs are allocated here unless
the caller gives them, raw device pointers and the current HIP stream go to the C ABI, and
a non-OK status raises ``FP4Error``.  What the C side cannot see is checked here: devices,
element types, shapes and contiguity.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch

from . import _lib as L

P, I32, I64, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class fp4_rmsnorm_desc(ctypes.Structure):
    _fields_ = [("rows", I64), ("cols", I64), ("x", P), ("ldx", I64), ("x_dtype", I32), ("terms", I32),
                ("term_weights", P), ("residual", P), ("ldr", I64), ("residual_out", P), ("ldro", I64),
                ("residual_dtype", I32), ("gamma_dtype", I32), ("gamma", P), ("eps", F32), ("y_dtype", I32), ("y", P),
                ("ldy", I64), ("grid", L.fp4_grid), ("gran", L.fp4_gran), ("tensor_scale", P), ("col_shift", P),
                ("packed", P), ("ldp", I64), ("scales", P)]


class fp4_swiglu8_desc(ctypes.Structure):
    _fields_ = [("rows", I64), ("cols", I64), ("x", P), ("ldx", I64), ("x_dtype", I32), ("reserved", I32),
                ("grid", L.fp4_grid), ("gran", L.fp4_gran), ("tensor_scale", P), ("col_shift", P), ("packed", P),
                ("ldp", I64), ("scales", P)]


class fp4_gemm_block_desc(ctypes.Structure):
    _fields_ = [("M", I64), ("N", I64), ("K", I64), ("a", P), ("lda", I64), ("a_scales", P), ("lda_s", I64),
                ("a_grid", L.fp4_grid), ("w", P), ("ldw", I64), ("w_scales", P), ("ldw_s", I64),
                ("w_grid", L.fp4_grid), ("y", P), ("ldy", I64), ("y_dtype", I32), ("reserved", I32)]


class fp4_route_desc(ctypes.Structure):
    _fields_ = [("tokens", I64), ("experts", I32), ("top_k", I32), ("logits", P), ("ld", I64), ("logits_dtype", I32),
                ("score", I32), ("bias", P), ("groups", I32), ("top_groups", I32), ("group_top", I32),
                ("renormalise", I32), ("scale", F32), ("reserved", I32), ("experts_out", P), ("weights_out", P),
                ("offsets", P), ("slots", P)]


class fp4_gemm_experts_desc(ctypes.Structure):
    _fields_ = [("slots", I64), ("N", I64), ("K", I64), ("experts", I32), ("slots_per_row", I32), ("a", P), ("lda", I64),
                ("a_scales", P), ("lda_s", I64), ("a_grid", L.fp4_grid), ("w", P), ("ldw", I64), ("stride_w", I64),
                ("w_scales", P), ("w_grid", L.fp4_grid), ("offsets", P), ("slot_list", P), ("y", P), ("ldy", I64),
                ("y_dtype", I32), ("reserved", I32)]


SIGNATURES = {
    "fp4_rmsnorm_quant": (I32, [ctypes.POINTER(fp4_rmsnorm_desc), P]),
    "fp4_swiglu_quant": (I32, [ctypes.POINTER(fp4_swiglu8_desc), P]),
    "fp4_quantize_block": (I32, [P, I32, I64, I64, I64, I64, I64, L.fp4_grid, P, I64, I64, P, P]),
    "fp4_gemm_block": (I32, [ctypes.POINTER(fp4_gemm_block_desc), P]),
    "fp4_route_workspace_size": (ctypes.c_size_t, [I64, I32, I32]),
    "fp4_route": (I32, [ctypes.POINTER(fp4_route_desc), P, ctypes.c_size_t, P]),
    "fp4_gemm_experts": (I32, [ctypes.POINTER(fp4_gemm_experts_desc), P]),
}

BLOCK = 128
_TYPES = {torch.float32: L.FP4_F32, torch.bfloat16: L.FP4_BF16}
_SCORES = {"softmax": 0, "sigmoid": 1}
_NO_GRID = L.fp4_grid()

Routing = namedtuple("Routing", "experts weights offsets slots")

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


def _type(t, name):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    return code


def _need(ok, message):
    if not ok:
        raise ValueError(message)


# The checks below run on every call, beside kernels of a few microseconds: one condition
# each, the message made only when it fails.
def _matrix(t, name, rows, cols, dev, dtype=None):
    """Leading dimension of the row-major [rows, cols] tensor t."""
    if t.shape != (rows, cols) or t.device != dev or (dtype is not None and t.dtype != dtype):
        raise ValueError(f"{name} must be [{rows}, {cols}]{f' {dtype}' if dtype else ''} on {dev}, "
                         f"not {list(t.shape)} {t.dtype} on {t.device}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must be row-major")
    return ld if rows > 1 or ld > cols else cols


def _flat(t, name, count, dtype, dev):
    """Pointer of a contiguous tensor of `count` values (None: 0)."""
    if t is None:
        return None
    if t.numel() != count or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} values on {dev}")
    return t.data_ptr()


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    """The current HIP stream of a device."""
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _check(status, func):
    if status:
        L.check(status, func)


def _units(g, rows, cols):
    return rows if g.mode == L.FP4_SCALE_ROW else rows * -(-cols // g.group) if g.mode == L.FP4_SCALE_GROUP and g.group > 0 else 0


def _code_output(g, rows, cols, dev, tensor_scale, col_shift, packed, scales):
    """The tail of a descriptor: tensor_scale, col_shift, packed, ldp, scales."""
    if packed is None:
        packed = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    kind = torch.float16 if g.scale_dtype == L.FP4_F16 else torch.float32
    if g.mode == L.FP4_SCALE_TENSOR:
        _need(scales is None, "scales are an output of row and group granularity only")
    elif scales is None:
        scales = torch.empty(_units(g, rows, cols), dtype=kind, device=dev)
    tail = (_flat(tensor_scale, "tensor_scale", 1, torch.float32, dev), _flat(col_shift, "col_shift", cols, torch.int8, dev),
            packed.data_ptr(), _matrix(packed, "packed", rows, cols, dev, torch.uint8),
            _flat(scales, "scales", _units(g, rows, cols), kind, dev))
    return packed, scales, tail


def fp4_rmsnorm_quant(x: torch.Tensor, gamma: torch.Tensor, grid: L.fp4_grid | None = None, g: L.fp4_gran | None = None,
                      eps: float = 1e-6, residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                      terms: int = 1, term_weights: torch.Tensor | None = None, tensor_scale: torch.Tensor | None = None,
                      col_shift: torch.Tensor | None = None, y: torch.Tensor | None = None,
                      packed: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """FP8 codes and scales of RMSNorm(residual + sum_j term_weights[:, j] x[terms r + j]) * gamma.

    x: [rows * terms, cols] f32 / bf16; term_weights: f32 [rows, terms].  residual_out (may
    be residual) takes the summed stream, y the normed rows.  Returns (packed, scales);
    without a grid no codes are made (y or residual_out must be given)."""
    _need(x.dim() == 2 and terms >= 1 and x.shape[0] % terms == 0, "x must be [rows * terms, cols]")
    rows, cols, dev = x.shape[0] // terms, x.shape[1], x.device
    tail = (None, None, None, 0, None)
    if grid is not None:
        _need(g is not None, "a grid needs a granularity")
        packed, scales, tail = _code_output(g, rows, cols, dev, tensor_scale, col_shift, packed, scales)
    else:
        _need(packed is None and scales is None, "packed and scales need a grid")
    stream = residual if residual is not None else residual_out
    if residual is not None and residual_out is not None:
        _need(residual.dtype == residual_out.dtype, "residual and residual_out must have one dtype")
    d = fp4_rmsnorm_desc(
        rows, cols, x.data_ptr(), _matrix(x, "x", rows * terms, cols, dev), _type(x, "x"), terms,
        _flat(term_weights, "term_weights", rows * terms, torch.float32, dev),
        residual.data_ptr() if residual is not None else None,
        _matrix(residual, "residual", rows, cols, dev) if residual is not None else 0,
        residual_out.data_ptr() if residual_out is not None else None,
        _matrix(residual_out, "residual_out", rows, cols, dev) if residual_out is not None else 0,
        _type(stream, "residual") if stream is not None else 0, _type(gamma, "gamma"),
        _flat(gamma, "gamma", cols, gamma.dtype, dev), eps, _type(y, "y") if y is not None else 0,
        y.data_ptr() if y is not None else None, _matrix(y, "y", rows, cols, dev) if y is not None else 0,
        grid if grid is not None else _NO_GRID, g if g is not None else L.fp4_gran(), *tail)
    _check(_call("fp4_rmsnorm_quant")(d, _stream(dev)), "fp4_rmsnorm_quant")
    return packed, scales


def fp4_swiglu_quant(x: torch.Tensor, grid: L.fp4_grid, g: L.fp4_gran, tensor_scale: torch.Tensor | None = None,
                     col_shift: torch.Tensor | None = None, packed: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None):
    """FP8 codes and scales of SiLU(x[:, :cols]) * x[:, cols:]; x: [rows, 2 cols] f32 / bf16.
    Returns (packed [rows, cols], scales)."""
    _need(x.dim() == 2 and x.shape[1] % 2 == 0, "x must be [rows, 2 cols]")
    rows, cols, dev = x.shape[0], x.shape[1] // 2, x.device
    packed, scales, tail = _code_output(g, rows, cols, dev, tensor_scale, col_shift, packed, scales)
    d = fp4_swiglu8_desc(rows, cols, x.data_ptr(), _matrix(x, "x", rows, 2 * cols, dev), _type(x, "x"), 0, grid, g, *tail)
    _check(_call("fp4_swiglu_quant")(d, _stream(dev)), "fp4_swiglu_quant")
    return packed, scales


def fp4_quantize_block(w: torch.Tensor, grid: L.fp4_grid, packed: torch.Tensor | None = None,
                       scales: torch.Tensor | None = None):
    """FP8 codes of w ([n, k] or [batch, n, k], f32 / bf16) with one f32 scale per 128 x 128
    block.  Returns (packed, scales [.., ceil(n / 128), ceil(k / 128)])."""
    _need(w.dim() in (2, 3), "w must be [n, k] or [batch, n, k]")
    lead, (n, k), dev = w.shape[:-2], w.shape[-2:], w.device
    blocks = (-(-n // BLOCK), -(-k // BLOCK))
    if packed is None:
        packed = torch.empty(w.shape, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((*lead, *blocks), dtype=torch.float32, device=dev)
    _need(packed.shape == w.shape and packed.dtype == torch.uint8 and packed.device == dev, "packed must be uint8 of w's shape")
    _need((w.stride(-1) == 1 and packed.stride(-1) == 1) or k <= 1, "w and packed must be row-major")
    ldw, ldp = (max(t.stride(-2), k) if n <= 1 else t.stride(-2) for t in (w, packed))
    batch = lead[0] if lead else 1
    _flat(scales, "scales", batch * blocks[0] * blocks[1], torch.float32, dev)
    _check(_call("fp4_quantize_block")(
        w.data_ptr(), _type(w, "w"), batch, n, k, ldw, w.stride(0) if lead else 0, grid, packed.data_ptr(),
        ldp, packed.stride(0) if lead else 0, scales.data_ptr(), _stream(dev)), "fp4_quantize_block")
    return packed, scales


def _a_scales(t, rows, K, dev):
    kb = -(-K // BLOCK)
    if t.dim() == 1:
        _flat(t, "a_scales", rows * kb, torch.float32, dev)
        return kb
    return _matrix(t, "a_scales", rows, kb, dev, torch.float32)


def fp4_gemm_block(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, a_grid: L.fp4_grid,
                   w_grid: L.fp4_grid, y_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None) -> torch.Tensor:
    """Y = X W^T of FP8 codes: a [M, K] with one f32 scale per row and 128 columns (flat, as
    the quantizers return them, or [M, ceil(K / 128)]), w [N, K] with one per 128 x 128."""
    _need(a.dim() == 2 and w.dim() == 2, "a must be [M, K], w [N, K]")
    (M, K), N, dev = a.shape, w.shape[0], a.device
    if y is None:
        y = torch.empty((M, N), dtype=y_dtype, device=dev)
    d = fp4_gemm_block_desc(
        M, N, K, a.data_ptr(), _matrix(a, "a", M, K, dev, torch.uint8), a_scales.data_ptr(), _a_scales(a_scales, M, K, dev),
        a_grid, w.data_ptr(), _matrix(w, "w", N, K, dev, torch.uint8), w_scales.data_ptr(),
        _matrix(w_scales, "w_scales", -(-N // BLOCK), -(-K // BLOCK), dev, torch.float32), w_grid, y.data_ptr(),
        _matrix(y, "y", M, N, dev), _type(y, "y"), 0)
    _check(_call("fp4_gemm_block")(d, _stream(dev)), "fp4_gemm_block")
    return y


def fp4_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None, groups: int = 1,
              top_groups: int = 1, group_top: int = 1, renormalise: bool = True, scale: float = 1.0, layout: bool = True,
              experts: torch.Tensor | None = None, weights: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
              slots: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> Routing:
    """The top_k experts of every token (logits [tokens, experts], f32 / bf16), their weights,
    and (layout) the slots token * top_k + j ordered by expert with each expert's offset.
    Logits that are infinite or NaN mark experts that the token may not use."""
    _need(logits.dim() == 2, "logits must be [tokens, experts]")
    (T, E), dev = logits.shape, logits.device
    if experts is None:
        experts = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    need = 0
    if layout:
        if offsets is None:
            offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
        if slots is None:
            slots = torch.empty(T * top_k, dtype=torch.int32, device=dev)
        need = _call("fp4_route_workspace_size")(T, E, top_k)
        if need and workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous memory on {dev}")
        if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        offsets = slots = None
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', not {score!r}")
    d = fp4_route_desc(
        T, E, top_k, logits.data_ptr(), _matrix(logits, "logits", T, E, dev), _type(logits, "logits"), _SCORES[score],
        _flat(bias, "bias", E, torch.float32, dev), groups, top_groups, group_top, int(bool(renormalise)), scale, 0,
        _flat(experts, "experts", T * top_k, torch.int32, dev), _flat(weights, "weights", T * top_k, torch.float32, dev),
        _flat(offsets, "offsets", E + 1, torch.int32, dev), _flat(slots, "slots", T * top_k, torch.int32, dev))
    _check(_call("fp4_route")(d, workspace.data_ptr() if need else None, need, _stream(dev)), "fp4_route")
    return Routing(experts, weights, offsets, slots)


def fp4_gemm_experts(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor, a_grid: L.fp4_grid,
                     w_grid: L.fp4_grid, offsets: torch.Tensor, slots: torch.Tensor, slots_per_row: int = 1,
                     y_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None) -> torch.Tensor:
    """Y[s] = X[s // slots_per_row] W[e]^T for the slots s that fp4_route's layout gives to
    expert e: a [rows, K] codes, w [experts, N, K] codes, scales as fp4_gemm_block.  Rows of
    y whose slot has no expert are not written (without y given, they hold zeros: all of it is
    cleared first, which takes 34 us for the 268 MB of 32768 x 4096 bf16)."""
    _need(a.dim() == 2 and w.dim() == 3, "a must be [rows, K], w [experts, N, K]")
    _need(slots_per_row >= 1 and slots.dim() == 1, "slots must be one list, slots_per_row positive")
    S, (E, N, K), dev = slots.shape[0], w.shape, a.device
    rows = -(-S // slots_per_row)
    if y is None:
        y = torch.zeros((S, N), dtype=y_dtype, device=dev)
    _need(w.dtype == torch.uint8 and w.device == dev and w.stride(2) == 1, "w must be row-major uint8 codes on a's device")
    d = fp4_gemm_experts_desc(
        S, N, K, E, slots_per_row, a.data_ptr(), _matrix(a, "a", rows, K, dev, torch.uint8), a_scales.data_ptr(),
        _a_scales(a_scales, rows, K, dev), a_grid, w.data_ptr(), w.stride(1), w.stride(0),
        _flat(w_scales, "w_scales", E * -(-N // BLOCK) * -(-K // BLOCK), torch.float32, dev), w_grid,
        _flat(offsets, "offsets", E + 1, torch.int32, dev), _flat(slots, "slots", S, torch.int32, dev), y.data_ptr(),
        _matrix(y, "y", S, N, dev), _type(y, "y"), 0)
    _check(_call("fp4_gemm_experts")(d, _stream(dev)), "fp4_gemm_experts")
    return y
