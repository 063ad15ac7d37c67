"""The layer operators: quantise, the product for any number of rows, routing, experts.

The same thin binding as the package's GEMV calls: ``nvfp4_*`` functions take
device pointers as integers, the functions without the prefix take torch tensors,
check them and allocate the outputs.  Every step of the computation runs in the
library's CUDA kernels; ``include/nvfp4_gemv.h`` defines each call.

There are no gradients (the weights are 4-bit codes): results are cut off from tensors that
require them, as under ``torch.no_grad()``.

``stream`` is a torch stream or a handle; None is the current one.  What a call on another
stream allocates is safe there and on the current stream; ordering the two streams, and
keeping the arguments until the call has run, is the caller's part.
"""
from __future__ import annotations

import ctypes

from . import (ACT_NONE, ACT_SILU, SF_PERMUTED_128x4, SF_PLAIN, _check, _empty as _empty_for, _need, _stream_handle,
               library)

DTYPE_FP16, DTYPE_BF16, DTYPE_FP32 = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class _GemmOptions(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("bias", ctypes.c_void_p), ("activation", ctypes.c_int32),
                ("c_dtype", ctypes.c_int32), ("c_row_stride", ctypes.c_int64)]


class _RouteOptions(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("weight_scale", ctypes.c_float)]


class _MoeOptions(ctypes.Structure):
    _fields_ = [("alpha1", ctypes.c_void_p), ("alpha2", ctypes.c_void_p), ("encode_x", ctypes.c_float),
                ("encode_h", ctypes.c_float), ("activation", ctypes.c_int32),
                ("round_outputs", ctypes.c_int32)]


class _MoeShape(ctypes.Structure):
    _fields_ = [("tile_rows", ctypes.c_int32), ("row_capacity", ctypes.c_int64),
                ("plan_bytes", ctypes.c_size_t)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the layer calls."""
    P, I64, I, F, Z = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    R = ctypes.POINTER
    for name, args in (
            ("nvfp4_quantize", [P, I, I64, I64, I64, I64, F, P, P, I, P, I, I64, P]),
            ("nvfp4_dequantize", [P, P, I, I64, I64, I64, F, P, I, I64, P]),
            ("nvfp4_fold_scale_signs", [P, P, I, I64, I64, I64, P]),
            ("nvfp4_gemm", [P, P, P, P, P, I64, I64, I64, I64, R(_GemmOptions), P]),
            ("nvfp4_gemm_plan", [I64, I64, I64, I64, I, R(I), R(I)]),
            ("nvfp4_route", [P, I, I64, I64, I64, I, R(_RouteOptions), P, P, P]),
            ("nvfp4_moe_shape", [I64, I64, I64, R(_MoeShape)]),
            ("nvfp4_moe_sort", [P, I64, I64, I64, P, P, P, P, P]),
            ("nvfp4_moe_gemm", [P, P, P, P, P, I64, I64, I64, I64, I64, P, I, P, I, P]),
            ("nvfp4_moe_gated_gemm", [P, P, P, P, P, I64, I64, I64, I64, I64, P, I, F, P, P, P]),
            ("nvfp4_moe_combine", [P, I, P, P, I64, I64, I64, P, I, P]),
            ("nvfp4_moe_ffn", [P, I, I64, P, P, P, P, P, P, I64, I64, I64, I64, I64, R(_MoeOptions), P, P, Z, P])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = I
    lib.nvfp4_moe_ffn_workspace_bytes.argtypes = [I64] * 5
    lib.nvfp4_moe_ffn_workspace_bytes.restype = Z


# ---------------------------------------------------------------------------
# device pointers
# ---------------------------------------------------------------------------

def nvfp4_quantize(x: int, x_dtype: int, rows: int, K: int, L: int, q: int, sf: int,
                   sf_layout: int = SF_PERMUTED_128x4, encode_scale: float = 1.0, x_row_stride: int = 0,
                   row_map: int = 0, copies: int = 0, q_rows: int = 0, stream: int = 0) -> None:
    """Enqueue the quantisation of x [L][rows][K]; with row_map, into the rows it names."""
    _check(library().nvfp4_quantize(x, x_dtype, x_row_stride, rows, K, L, encode_scale, q, sf, sf_layout,
                                    row_map or None, copies, q_rows, stream), "nvfp4_quantize")


def nvfp4_dequantize(q: int, sf: int, rows: int, K: int, L: int, x: int, x_dtype: int,
                     sf_layout: int = SF_PERMUTED_128x4, scale: float = 1.0, x_row_stride: int = 0,
                     stream: int = 0) -> None:
    """Enqueue x [L][rows][K] = the values of q and sf, times scale."""
    _check(library().nvfp4_dequantize(q, sf, sf_layout, rows, K, L, scale, x, x_dtype, x_row_stride, stream),
           "nvfp4_dequantize")


def nvfp4_fold_scale_signs(a: int, sf: int, rows: int, K: int, L: int, sf_layout: int = SF_PERMUTED_128x4,
                           stream: int = 0) -> None:
    """Move the scales' signs into the elements, in place."""
    _check(library().nvfp4_fold_scale_signs(a, sf, sf_layout, rows, K, L, stream), "nvfp4_fold_scale_signs")


def nvfp4_gemm(a: int, b: int, sfa: int, sfb: int, c: int, M: int, N: int, K: int, L: int, alpha: float = 1.0,
               bias: int = 0, activation: int = ACT_NONE, c_dtype: int = DTYPE_FP16, c_row_stride: int = 0,
               stream: int = 0) -> None:
    """Enqueue c [L][N][M] = act(alpha * a b + bias) for quantised a [L][M], b [L][N]; the scales'
    signs are ignored."""
    opt = _GemmOptions(alpha, bias or None, activation, c_dtype, c_row_stride)
    _check(library().nvfp4_gemm(a, b, sfa, sfb, c, M, N, K, L, ctypes.byref(opt), stream), "nvfp4_gemm")


def nvfp4_gemm_plan(M: int, N: int, K: int, L: int = 1, num_sms: int = 152) -> dict:
    """The tile and K split that nvfp4_gemm uses without an activation (host only)."""
    rows, split = ctypes.c_int(), ctypes.c_int()
    _check(library().nvfp4_gemm_plan(M, N, K, L, num_sms, ctypes.byref(rows), ctypes.byref(split)),
           "nvfp4_gemm_plan")
    return {"tile_rows": rows.value, "k_split": split.value}


def nvfp4_route(logits: int, dtype: int, T: int, E: int, top_k: int, ids: int, weights: int,
                score: int = SCORE_SOFTMAX, bias: int = 0, groups: int = 1, top_groups: int = 1,
                renormalize: bool = True, weight_scale: float = 1.0, row_stride: int = 0,
                stream: int = 0) -> None:
    """Enqueue the choice of top_k of E experts for T tokens."""
    opt = _RouteOptions(score, bias or None, groups, top_groups, 1 if renormalize else 0, weight_scale)
    _check(library().nvfp4_route(logits, dtype, row_stride, T, E, top_k, ctypes.byref(opt), ids, weights,
                                 stream), "nvfp4_route")


def nvfp4_moe_shape(T: int, top_k: int, E: int) -> dict:
    """Tile, row capacity and plan size of the experts' rows (host only)."""
    s = _MoeShape()
    _check(library().nvfp4_moe_shape(T, top_k, E, ctypes.byref(s)), "nvfp4_moe_shape")
    return {"tile_rows": s.tile_rows, "row_capacity": s.row_capacity, "plan_bytes": s.plan_bytes}


def nvfp4_moe_sort(ids: int, T: int, top_k: int, E: int, rows: int, counts: int, starts: int, plan: int,
                   stream: int = 0) -> None:
    """Enqueue the sort of the choices by expert."""
    _check(library().nvfp4_moe_sort(ids, T, top_k, E, rows, counts, starts, plan, stream), "nvfp4_moe_sort")


def nvfp4_moe_gemm(a: int, sfa: int, b: int, sfb: int, plan: int, T: int, top_k: int, E: int, M: int, K: int,
                   c: int, c_dtype: int, alpha: int = 0, activation: int = ACT_NONE, stream: int = 0) -> None:
    """Enqueue the experts' product of their rows."""
    _check(library().nvfp4_moe_gemm(a, sfa, b, sfb, plan, T, top_k, E, M, K, alpha or None, activation, c,
                                    c_dtype, stream), "nvfp4_moe_gemm")


def nvfp4_moe_gated_gemm(a: int, sfa: int, b: int, sfb: int, plan: int, T: int, top_k: int, E: int, F: int,
                         K: int, q: int, sf: int, alpha: int = 0, activation: int = ACT_SILU,
                         encode_scale: float = 1.0, stream: int = 0) -> None:
    """Enqueue the experts' gated product with a quantised result."""
    _check(library().nvfp4_moe_gated_gemm(a, sfa, b, sfb, plan, T, top_k, E, F, K, alpha or None, activation,
                                          encode_scale, q, sf, stream), "nvfp4_moe_gated_gemm")


def nvfp4_moe_combine(y: int, y_dtype: int, rows: int, weights: int, T: int, top_k: int, M: int, out: int,
                      dtype: int, stream: int = 0) -> None:
    """Enqueue the weighted sum of each token's rows."""
    _check(library().nvfp4_moe_combine(y, y_dtype, rows, weights, T, top_k, M, out, dtype, stream),
           "nvfp4_moe_combine")


def nvfp4_moe_ffn_workspace_bytes(T: int, top_k: int, E: int, D: int, F: int) -> int:
    return int(library().nvfp4_moe_ffn_workspace_bytes(T, top_k, E, D, F))


def nvfp4_moe_ffn(x: int, dtype: int, ids: int, weights: int, w1: int, sf1: int, w2: int, sf2: int, T: int,
                  top_k: int, E: int, D: int, F: int, out: int, workspace: int, workspace_bytes: int,
                  alpha1: int = 0, alpha2: int = 0, encode_x: float = 1.0, encode_h: float = 1.0,
                  activation: int = ACT_SILU, x_row_stride: int = 0, stream: int = 0,
                  round_outputs: bool = False) -> None:
    """Enqueue the routed feed-forward layer."""
    opt = _MoeOptions(alpha1 or None, alpha2 or None, encode_x, encode_h, activation, 1 if round_outputs else 0)
    _check(library().nvfp4_moe_ffn(x, dtype, x_row_stride, ids, weights, w1, sf1, w2, sf2, T, top_k, E, D, F,
                                   ctypes.byref(opt), out, workspace, workspace_bytes, stream),
           "nvfp4_moe_ffn")


# ---------------------------------------------------------------------------
# torch tensors
# ---------------------------------------------------------------------------
# A call that decodes one token spends more time here than on the GPU, so these
# make their checks in few steps: _ptr looks at everything _need looks at and
# leaves the message to it, and _enqueue enters a device context only when
# another device is current.

_torch = None
_codes = {}


def _load():
    """torch, imported at the first call (the device-pointer functions do without)."""
    global _torch
    if _torch is None:
        import torch

        _codes.update({torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32})
        _torch = torch
    return _torch


def _ptr(t, name, dtype, numel, device) -> int:
    """The address of a contiguous tensor of this type, size and device."""
    try:
        if t.dtype is dtype and t.numel() == numel and t.is_contiguous() and (
                t.get_device() == device.index or not numel):
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, name, dtype, numel, device)
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=device)
    return _empty_for(shape, dtype, device, stream)


def _dtype_code(x, name, fp32=True) -> int:
    code = _codes.get(getattr(x, "dtype", x))
    if code is None or (code == DTYPE_FP32 and not fp32):
        allowed = "float16, bfloat16 or float32" if fp32 else "float16 or bfloat16"
        raise TypeError(f"{name} must be {allowed}, got {getattr(x, 'dtype', x)}")
    return code


def _rows(x, name):
    """A matrix whose rows are contiguous: rows, columns, row stride."""
    if x.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, has {x.dim()}")
    n, k = x.shape
    stride, step = x.stride()
    if k > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if n > 1 and stride < k:
        raise ValueError(f"{name} must have rows that do not overlap")
    return n, k, stride if n > 1 else k


def _enqueue(where, device, stream, *args) -> None:
    """The library's call `where` on args and the stream, with `device` current."""
    index = device.index
    if index is None:
        raise ValueError(f"the tensors are on {device}, expected a CUDA device")
    handle = _torch._C._cuda_getCurrentRawStream(index) if stream is None else _stream_handle(stream, device)
    call = getattr(library(), where)
    if index == _torch._C._cuda_getDevice():
        status = call(*args, handle)
    else:
        with _torch.cuda.device(index):
            status = call(*args, handle)
    if status:
        _check(status, where)


def _scale_bytes(layout, rows, K, L):
    if layout == SF_PLAIN:
        return L * rows * (K // 16)
    return L * ((rows + 127) // 128) * ((K + 63) // 64) * 512


def quantize(x, encode_scale: float = 1.0, sf_layout: int = SF_PERMUTED_128x4, q=None, sf=None, stream=None):
    """(q uint8 [rows, K//2], sf uint8 flat) of x [rows, K] (fp16, bf16 or fp32, rows may be
    strided); a 3-d contiguous x [L, rows, K] gives q [L, rows, K//2] and scales per batch."""
    torch = _torch or _load()
    code = _dtype_code(x, "x")
    if x.dim() == 3:
        _ptr(x, "x", x.dtype, x.numel(), x.device)
        (L, rows, K), stride = x.shape, 0
    else:
        L, (rows, K, stride) = 1, _rows(x, "x")
    if K % 16:
        raise ValueError(f"x has rows of {K} elements, expected a multiple of 16")
    n, dev, u8 = _scale_bytes(sf_layout, rows, K, L), x.device, torch.uint8
    if q is None:
        q = _empty((rows, K // 2) if x.dim() == 2 else (L, rows, K // 2), u8, dev, stream)
    else:
        _ptr(q, "q", u8, L * rows * (K // 2), dev)
    if sf is None:
        sf = _empty(n, u8, dev, stream)
    else:
        _ptr(sf, "sf", u8, n, dev)
    _enqueue("nvfp4_quantize", dev, stream, x.data_ptr(), code, stride, rows, K, L, encode_scale, q.data_ptr(),
             sf.data_ptr(), sf_layout, None, 0, 0)
    return q, sf


def dequantize(q, sf, scale: float = 1.0, dtype=None, sf_layout: int = SF_PERMUTED_128x4, x=None, stream=None):
    """The values of q [..., rows, K//2] and sf, times scale, as dtype (default float32)."""
    torch = _torch or _load()
    shape, dev, u8 = q.shape, q.device, torch.uint8
    if len(shape) not in (2, 3):
        raise ValueError("q must be [rows, K//2] or [L, rows, K//2]")
    L, rows, half = shape if len(shape) == 3 else (1, *shape)
    K = 2 * half
    if K % 16:
        raise ValueError(f"q has rows of {K} elements, expected a multiple of 16")
    if dtype is None:
        dtype = torch.float32 if x is None else x.dtype
    code = _dtype_code(dtype, "dtype")
    qp = _ptr(q, "q", u8, L * rows * (K // 2), dev)
    sp = _ptr(sf, "sf", u8, _scale_bytes(sf_layout, rows, K, L), dev)
    if x is None:
        x = _empty((rows, K) if len(shape) == 2 else (L, rows, K), dtype, dev, stream)
    else:
        _ptr(x, "x", dtype, L * rows * K, dev)
    _enqueue("nvfp4_dequantize", dev, stream, qp, sp, sf_layout, rows, K, L, scale, x.data_ptr(), code, 0)
    return x


def fold_scale_signs(a, sf, sf_layout: int = SF_PERMUTED_128x4, stream=None):
    """Make the scales of a [L, rows, K//2] unsigned, in place; returns (a, sf)."""
    torch = _torch or _load()
    if a.dim() != 3:
        raise ValueError("a must be [L, rows, K//2]")
    L, rows, K = a.shape[0], a.shape[1], 2 * a.shape[2]
    if K % 16:
        raise ValueError(f"a has rows of {K} elements, expected a multiple of 16")
    _enqueue("nvfp4_fold_scale_signs", a.device, stream, _ptr(a, "a", torch.uint8, a.numel(), a.device),
             _ptr(sf, "sf", torch.uint8, _scale_bytes(sf_layout, rows, K, L), a.device), sf_layout, rows, K, L)
    return a, sf


def gemm(a, b, sfa, sfb, alpha: float = 1.0, bias=None, activation: int = ACT_NONE, dtype=None, c=None,
         stream=None):
    """c [L, N, M] = act(alpha * b a^T + bias) from a [L, M, K//2], b [L, N, K//2] (uint8) and their
    permuted scales (flat uint8); bias fp32 [L, M]; dtype float16 (default), bfloat16 or float32.
    The scales are read as magnitudes, their signs ignored, unlike gemv() and nvfp4_gemm_small_n():
    fold_scale_signs() makes signed ones unsigned, once.  For a single row nvfp4_gemm_small_n() is
    the faster call, for 2 to 16 this one."""
    torch = _torch or _load()
    ashape, bshape = a.shape, b.shape
    if len(ashape) != 3 or len(bshape) != 3 or ashape[0] != bshape[0] or ashape[2] != bshape[2]:
        raise ValueError("a must be [L, M, K//2] and b [L, N, K//2]")
    L, M, half_k = ashape
    N, K, dev, u8 = bshape[1], 2 * half_k, a.device, torch.uint8
    if K % 16:
        raise ValueError(f"a has rows of {K} elements, expected a multiple of 16")
    ap, bp = _ptr(a, "a", u8, L * M * half_k, dev), _ptr(b, "b", u8, L * N * half_k, dev)
    sap = _ptr(sfa, "sfa", u8, _scale_bytes(SF_PERMUTED_128x4, M, K, L), dev)
    sbp = _ptr(sfb, "sfb", u8, _scale_bytes(SF_PERMUTED_128x4, N, K, L), dev)
    bias_p = None if bias is None else _ptr(bias, "bias", torch.float32, L * M, dev)
    if dtype is None:
        dtype = torch.float16 if c is None else c.dtype
    code = _dtype_code(dtype, "dtype")
    if c is None:
        c = _empty((L, N, M), dtype, dev, stream)
    else:
        _ptr(c, "c", dtype, L * N * M, dev)
    _enqueue("nvfp4_gemm", dev, stream, ap, bp, sap, sbp, c.data_ptr(), M, N, K, L,
             ctypes.byref(_GemmOptions(alpha, bias_p, activation, code, 0)))
    return c


def route(logits, top_k: int, score: int = SCORE_SOFTMAX, bias=None, groups: int = 1, top_groups: int = 1,
          renormalize: bool = True, weight_scale: float = 1.0, stream=None):
    """(ids int32 [T, top_k], weights fp32 [T, top_k]) of logits [T, E]; no gradients."""
    torch = _torch or _load()
    code = _dtype_code(logits, "logits")
    T, E, stride = _rows(logits, "logits")
    dev = logits.device
    bias_p = None if bias is None else _ptr(bias, "bias", torch.float32, E, dev)
    ids = _empty((T, top_k), torch.int32, dev, stream)
    weights = _empty((T, top_k), torch.float32, dev, stream)
    _enqueue("nvfp4_route", dev, stream, logits.data_ptr(), code, stride, T, E, top_k,
             ctypes.byref(_RouteOptions(score, bias_p, groups, top_groups, 1 if renormalize else 0, weight_scale)),
             ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_sort(ids, E: int, stream=None) -> dict:
    """Sort the choices ids [T, top_k] (int32) by expert: rows [T, top_k], counts [E], starts [E],
    the plan of the products and the capacity and tile of the experts' rows."""
    torch = _torch or _load()
    if ids.dim() != 2:
        raise ValueError("ids must be [T, top_k]")
    (T, k), dev, i32 = ids.shape, ids.device, torch.int32
    p = _ptr(ids, "ids", i32, T * k, dev)
    shape = nvfp4_moe_shape(T, k, E)
    out = {"rows": _empty((T, k), i32, dev, stream), "counts": _empty(E, i32, dev, stream),
           "starts": _empty(E, i32, dev, stream),
           "plan": _empty(shape["plan_bytes"], torch.uint8, dev, stream),
           "row_capacity": shape["row_capacity"], "tile_rows": shape["tile_rows"], "experts": E}
    _enqueue("nvfp4_moe_sort", dev, stream, p, T, k, E, out["rows"].data_ptr(), out["counts"].data_ptr(),
             out["starts"].data_ptr(), out["plan"].data_ptr())
    return out


def _need_sorted(order, b, sfb, dev):
    torch = _torch or _load()
    T, k = order["rows"].shape
    E, rows = order["experts"], order["row_capacity"]
    _need(order["plan"], "plan", torch.uint8, nvfp4_moe_shape(T, k, E)["plan_bytes"], dev)
    if b.dim() != 2:
        raise ValueError("b must be [row_capacity, K//2]")
    K = 2 * b.shape[1]
    if K % 32:
        raise ValueError(f"b has rows of {K} elements, expected a multiple of 32")
    _need(b, "b", torch.uint8, rows * (K // 2), dev)
    _need(sfb, "sfb", torch.uint8, _scale_bytes(SF_PERMUTED_128x4, rows, K, 1), dev)
    return T, k, E, rows, K


def _need_experts(a, sfa, alpha, E, K, dev):
    """(M, and the addresses of the weights, their scales and alpha)."""
    torch = _torch or _load()
    if a.dim() != 3 or a.shape[0] != E or 2 * a.shape[2] != K:
        raise ValueError(f"the weights must be [{E}, M, {K // 2}]")
    M = a.shape[1]
    return (M, _ptr(a, "weights", torch.uint8, E * M * (K // 2), dev),
            _ptr(sfa, "weight scales", torch.uint8, _scale_bytes(SF_PERMUTED_128x4, M, K, E), dev),
            None if alpha is None else _ptr(alpha, "alpha", torch.float32, E, dev))


def quantize_rows(x, order, encode_scale: float = 1.0, stream=None):
    """Quantise the tokens x [T, K] into the experts' rows of a moe_sort."""
    torch = _torch or _load()
    code = _dtype_code(x, "x")
    T, K, stride = _rows(x, "x")
    dev, rows, k = x.device, order["row_capacity"], order["rows"].shape[1]
    if K % 16:
        raise ValueError(f"x has rows of {K} elements, expected a multiple of 16")
    to = _ptr(order["rows"], "rows", torch.int32, T * k, dev)
    q = _empty((rows, K // 2), torch.uint8, dev, stream)
    sf = _empty(_scale_bytes(SF_PERMUTED_128x4, rows, K, 1), torch.uint8, dev, stream)
    _enqueue("nvfp4_quantize", dev, stream, x.data_ptr(), code, stride, T, K, 1, encode_scale, q.data_ptr(),
             sf.data_ptr(), SF_PERMUTED_128x4, to, k, rows)
    return q, sf


def moe_gemm(a, sfa, b, sfb, order, alpha=None, activation: int = ACT_NONE, dtype=None, stream=None):
    """c [row_capacity, M] = act(alpha[e] * b a[e]^T) for the experts' rows b of a moe_sort."""
    torch = _torch or _load()
    dev = a.device
    T, k, E, rows, K = _need_sorted(order, b, sfb, dev)
    M, ap, sp, alpha_p = _need_experts(a, sfa, alpha, E, K, dev)
    dtype = dtype or torch.float16
    code = _dtype_code(dtype, "dtype")
    c = _empty((rows, M), dtype, dev, stream)
    _enqueue("nvfp4_moe_gemm", dev, stream, ap, sp, b.data_ptr(), sfb.data_ptr(), order["plan"].data_ptr(), T, k,
             E, M, K, alpha_p, activation, c.data_ptr(), code)
    return c


def moe_gated_gemm(a, sfa, b, sfb, order, alpha=None, activation: int = ACT_SILU, encode_scale: float = 1.0,
                   stream=None):
    """(q [row_capacity, F//2], sf) of act(gate) * input, gate and input the even and odd rows of
    a [E, 2F, K//2], for the experts' rows b of a moe_sort."""
    torch = _torch or _load()
    dev = a.device
    T, k, E, rows, K = _need_sorted(order, b, sfb, dev)
    M, ap, sp, alpha_p = _need_experts(a, sfa, alpha, E, K, dev)
    if M % 64:
        raise ValueError(f"the weights have {M} rows, expected a multiple of 64")
    F = M // 2
    q = _empty((rows, F // 2), torch.uint8, dev, stream)
    sf = _empty(_scale_bytes(SF_PERMUTED_128x4, rows, F, 1), torch.uint8, dev, stream)
    _enqueue("nvfp4_moe_gated_gemm", dev, stream, ap, sp, b.data_ptr(), sfb.data_ptr(), order["plan"].data_ptr(),
             T, k, E, F, K, alpha_p, activation, encode_scale, q.data_ptr(), sf.data_ptr())
    return q, sf


def moe_combine(y, order, weights, dtype=None, stream=None):
    """out [T, M] = sum_j weights[t, j] * y[rows[t, j]], as dtype (fp16 or bf16; y's own, or y in
    float32)."""
    torch = _torch or _load()
    y_code = _dtype_code(y, "y")
    dtype = dtype or y.dtype
    code = _dtype_code(dtype, "dtype", fp32=False)
    if y.dim() != 2:
        raise ValueError("y must be [row_capacity, M]")
    T, k = order["rows"].shape
    M, dev = y.shape[1], y.device
    yp = _ptr(y, "y", y.dtype, order["row_capacity"] * M, dev)
    wp = _ptr(weights, "weights", torch.float32, T * k, dev)
    out = _empty((T, M), dtype, dev, stream)
    _enqueue("nvfp4_moe_combine", dev, stream, yp, y_code, order["rows"].data_ptr(), wp, T, k, M, out.data_ptr(),
             code)
    return out


def moe_ffn(x, ids, weights, w1, sf1, w2, sf2, alpha1=None, alpha2=None, encode_x: float = 1.0,
            encode_h: float = 1.0, activation: int = ACT_SILU, out=None, workspace=None, stream=None,
            round_outputs: bool = False):
    """The routed feed-forward layer: out [T, D] from x [T, D] (fp16 or bf16), ids and weights
    [T, top_k], w1 [E, 2F, D//2] (gate and input rows interleaved), w2 [E, D, F//2] and their
    permuted scales.  workspace: a uint8 tensor of nvfp4_moe_ffn_workspace_bytes, or None.
    round_outputs: the experts' outputs are rounded to the type of x before the weighted sum
    (fewer bytes in large batches) in place of being held in fp32.  No gradients."""
    torch = _torch or _load()
    code = _dtype_code(x, "x", fp32=False)
    T, D, stride = _rows(x, "x")
    dev = x.device
    if ids.dim() != 2:
        raise ValueError("ids must be [T, top_k]")
    k = ids.shape[1]
    idp = _ptr(ids, "ids", torch.int32, T * k, dev)
    wp = _ptr(weights, "weights", torch.float32, T * k, dev)
    shape1, shape2 = w1.shape, w2.shape
    if len(shape1) != 3 or len(shape2) != 3:
        raise ValueError("w1 must be [E, 2F, D//2] and w2 [E, D, F//2]")
    E, F = shape1[0], 2 * shape2[2]
    if shape1 != (E, 2 * F, D // 2) or shape2 != (E, D, F // 2) or D % 32 or F % 32:
        raise ValueError("w1 must be [E, 2F, D//2] and w2 [E, D, F//2], D and F multiples of 32")
    u8, f32 = torch.uint8, torch.float32
    p1, p2 = _ptr(w1, "w1", u8, E * F * D, dev), _ptr(w2, "w2", u8, E * D * (F // 2), dev)
    s1 = _ptr(sf1, "sf1", u8, _scale_bytes(SF_PERMUTED_128x4, 2 * F, D, E), dev)
    s2 = _ptr(sf2, "sf2", u8, _scale_bytes(SF_PERMUTED_128x4, D, F, E), dev)
    a1 = None if alpha1 is None else _ptr(alpha1, "alpha1", f32, E, dev)
    a2 = None if alpha2 is None else _ptr(alpha2, "alpha2", f32, E, dev)
    if out is None:
        out = _empty((T, D), x.dtype, dev, stream)
    else:
        _ptr(out, "out", x.dtype, T * D, dev)
    need = library().nvfp4_moe_ffn_workspace_bytes(T, k, E, D, F)
    if workspace is None:
        workspace, size = _empty(need, u8, dev, stream), need
    else:
        size = workspace.numel()
        if size < need:
            raise ValueError(f"workspace has {size} bytes, expected {need}")
        _ptr(workspace, "workspace", u8, size, dev)
    _enqueue("nvfp4_moe_ffn", dev, stream, x.data_ptr(), code, stride, idp, wp, p1, s1, p2, s2, T, k, E, D, F,
             ctypes.byref(_MoeOptions(a1, a2, encode_x, encode_h, activation, 1 if round_outputs else 0)),
             out.data_ptr(), workspace.data_ptr(), size)
    return out
