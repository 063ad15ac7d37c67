"""The layer operators: quantise, the product for any number of rows, routing, experts.

The same thin binding as the package's GEMV calls: ``nvfp4_*`` functions take
device pointers as integers, the functions without the prefix take torch tensors,
check them and allocate the outputs.  Every step of the computation runs in the
library's CUDA kernels; ``include/nvfp4_gemv.h`` defines each call.
"""
from __future__ import annotations

import ctypes

from . import (ACT_NONE, ACT_SILU, SF_PERMUTED_128x4, SF_PLAIN, _check, _need, _on_device, _stream_handle,
               library, nvfp4_permuted_scale_bytes)

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
                ("encode_h", ctypes.c_float), ("activation", ctypes.c_int32)]


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
            ("nvfp4_route", [P, I, I64, I64, I64, I, R(_RouteOptions), P, P, P]),
            ("nvfp4_moe_shape", [I64, I64, I64, R(_MoeShape)]),
            ("nvfp4_moe_sort", [P, I64, I64, I64, P, P, P, P, P]),
            ("nvfp4_moe_gemm", [P, P, P, P, P, I64, I64, I64, I64, I64, P, I, P, I, P]),
            ("nvfp4_moe_gated_gemm", [P, P, P, P, P, I64, I64, I64, I64, I64, P, I, F, P, P, P]),
            ("nvfp4_moe_combine", [P, I, P, P, I64, I64, I64, P, P]),
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
    """Enqueue c [L][N][M] = act(alpha * a b + bias) for quantised a [L][M], b [L][N]."""
    opt = _GemmOptions(alpha, bias or None, activation, c_dtype, c_row_stride)
    _check(library().nvfp4_gemm(a, b, sfa, sfb, c, M, N, K, L, ctypes.byref(opt), stream), "nvfp4_gemm")


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


def nvfp4_moe_combine(y: int, dtype: int, rows: int, weights: int, T: int, top_k: int, M: int, out: int,
                      stream: int = 0) -> None:
    """Enqueue the weighted sum of each token's rows."""
    _check(library().nvfp4_moe_combine(y, dtype, rows, weights, T, top_k, M, out, stream), "nvfp4_moe_combine")


def nvfp4_moe_ffn_workspace_bytes(T: int, top_k: int, E: int, D: int, F: int) -> int:
    return int(library().nvfp4_moe_ffn_workspace_bytes(T, top_k, E, D, F))


def nvfp4_moe_ffn(x: int, dtype: int, ids: int, weights: int, w1: int, sf1: int, w2: int, sf2: int, T: int,
                  top_k: int, E: int, D: int, F: int, out: int, workspace: int, workspace_bytes: int,
                  alpha1: int = 0, alpha2: int = 0, encode_x: float = 1.0, encode_h: float = 1.0,
                  activation: int = ACT_SILU, x_row_stride: int = 0, stream: int = 0) -> None:
    """Enqueue the routed feed-forward layer."""
    opt = _MoeOptions(alpha1 or None, alpha2 or None, encode_x, encode_h, activation)
    _check(library().nvfp4_moe_ffn(x, dtype, x_row_stride, ids, weights, w1, sf1, w2, sf2, T, top_k, E, D, F,
                                   ctypes.byref(opt), out, workspace, workspace_bytes, stream),
           "nvfp4_moe_ffn")


# ---------------------------------------------------------------------------
# torch tensors
# ---------------------------------------------------------------------------

def _dtype_code(dtype, name, allowed=("float16", "bfloat16", "float32")) -> int:
    import torch

    codes = {torch.float16: DTYPE_FP16, torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_FP32}
    if dtype not in codes or str(dtype).split(".")[-1] not in allowed:
        raise TypeError(f"{name} must be one of {', '.join(allowed)}, got {dtype}")
    return codes[dtype]


def _need_rows(x, name):
    """A matrix whose rows are contiguous; returns its row stride."""
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, has {x.dim()}")
    if x.shape[1] > 1 and x.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if x.shape[0] > 1 and x.stride(0) < x.shape[1]:
        raise ValueError(f"{name} must have rows that do not overlap")
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _on_gpu(device):
    """_on_device for a call that reads tensors: they have to be on a GPU."""
    if device.type != "cuda":
        raise ValueError(f"the tensors are on {device}, expected a CUDA device")
    return _on_device(device)


def _scale_bytes(layout, rows, K, L):
    return L * rows * (K // 16) if layout == SF_PLAIN else nvfp4_permuted_scale_bytes(rows, K, L)


def quantize(x, encode_scale: float = 1.0, sf_layout: int = SF_PERMUTED_128x4, q=None, sf=None, stream=None):
    """(q uint8 [rows, K//2], sf uint8 flat) of x [rows, K] (fp16, bf16 or fp32, rows may be
    strided); a 3-d contiguous x [L, rows, K] gives q [L, rows, K//2] and scales per batch."""
    import torch

    code = _dtype_code(getattr(x, "dtype", None), "x")
    if x.dim() == 3:
        _need(x, "x", x.dtype, x.numel(), x.device)
        (L, rows, K), stride = x.shape, 0
    else:
        stride = _need_rows(x, "x")
        L, (rows, K) = 1, x.shape
    if K % 16:
        raise ValueError(f"x has rows of {K} elements, expected a multiple of 16")
    n = _scale_bytes(sf_layout, rows, K, L)
    if q is None:
        q = torch.empty((*x.shape[:-1], K // 2), dtype=torch.uint8, device=x.device)
    if sf is None:
        sf = torch.empty(n, dtype=torch.uint8, device=x.device)
    _need(q, "q", torch.uint8, L * rows * (K // 2), x.device)
    _need(sf, "sf", torch.uint8, n, x.device)
    with _on_gpu(x.device):
        nvfp4_quantize(x.data_ptr(), code, rows, K, L, q.data_ptr(), sf.data_ptr(), sf_layout, encode_scale,
                       stride, stream=_stream_handle(stream, x.device))
    return q, sf


def dequantize(q, sf, scale: float = 1.0, dtype=None, sf_layout: int = SF_PERMUTED_128x4, x=None, stream=None):
    """The values of q [..., rows, K//2] and sf, times scale, as dtype (default float32)."""
    import torch

    if q.dim() not in (2, 3):
        raise ValueError("q must be [rows, K//2] or [L, rows, K//2]")
    L = q.shape[0] if q.dim() == 3 else 1
    rows, K = q.shape[-2], 2 * q.shape[-1]
    if K % 16:
        raise ValueError(f"q has rows of {K} elements, expected a multiple of 16")
    dtype = dtype or (torch.float32 if x is None else x.dtype)
    code = _dtype_code(dtype, "dtype")
    _need(q, "q", torch.uint8, L * rows * (K // 2), q.device)
    _need(sf, "sf", torch.uint8, _scale_bytes(sf_layout, rows, K, L), q.device)
    if x is None:
        x = torch.empty((*q.shape[:-1], K), dtype=dtype, device=q.device)
    _need(x, "x", dtype, L * rows * K, q.device)
    with _on_gpu(q.device):
        nvfp4_dequantize(q.data_ptr(), sf.data_ptr(), rows, K, L, x.data_ptr(), code, sf_layout, scale,
                         stream=_stream_handle(stream, q.device))
    return x


def fold_scale_signs(a, sf, sf_layout: int = SF_PERMUTED_128x4, stream=None):
    """Make the scales of a [L, rows, K//2] unsigned, in place; returns (a, sf)."""
    import torch

    if a.dim() != 3:
        raise ValueError("a must be [L, rows, K//2]")
    L, rows, K = a.shape[0], a.shape[1], 2 * a.shape[2]
    if K % 16:
        raise ValueError(f"a has rows of {K} elements, expected a multiple of 16")
    _need(a, "a", torch.uint8, a.numel(), a.device)
    _need(sf, "sf", torch.uint8, _scale_bytes(sf_layout, rows, K, L), a.device)
    with _on_gpu(a.device):
        nvfp4_fold_scale_signs(a.data_ptr(), sf.data_ptr(), rows, K, L, sf_layout,
                               _stream_handle(stream, a.device))
    return a, sf


def gemm(a, b, sfa, sfb, alpha: float = 1.0, bias=None, activation: int = ACT_NONE, dtype=None, c=None,
         stream=None):
    """c [L, N, M] = act(alpha * b a^T + bias) from a [L, M, K//2], b [L, N, K//2] (uint8) and their
    permuted scales (flat uint8); bias fp32 [L, M]; dtype float16 (default), bfloat16 or float32."""
    import torch

    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[2] != b.shape[2]:
        raise ValueError("a must be [L, M, K//2] and b [L, N, K//2]")
    L, M, half_k = a.shape
    N, K, dev = b.shape[1], 2 * half_k, a.device
    if K % 16:
        raise ValueError(f"a has rows of {K} elements, expected a multiple of 16")
    _need(a, "a", torch.uint8, L * M * half_k, dev)
    _need(b, "b", torch.uint8, L * N * half_k, dev)
    _need(sfa, "sfa", torch.uint8, nvfp4_permuted_scale_bytes(M, K, L), dev)
    _need(sfb, "sfb", torch.uint8, nvfp4_permuted_scale_bytes(N, K, L), dev)
    if bias is not None:
        _need(bias, "bias", torch.float32, L * M, dev)
    dtype = dtype or (torch.float16 if c is None else c.dtype)
    code = _dtype_code(dtype, "dtype")
    if c is None:
        c = torch.empty((L, N, M), dtype=dtype, device=dev)
    _need(c, "c", dtype, L * N * M, dev)
    with _on_gpu(dev):
        nvfp4_gemm(a.data_ptr(), b.data_ptr(), sfa.data_ptr(), sfb.data_ptr(), c.data_ptr(), M, N, K, L, alpha,
                   bias.data_ptr() if bias is not None else 0, activation, code,
                   stream=_stream_handle(stream, dev))
    return c


def route(logits, top_k: int, score: int = SCORE_SOFTMAX, bias=None, groups: int = 1, top_groups: int = 1,
          renormalize: bool = True, weight_scale: float = 1.0, stream=None):
    """(ids int32 [T, top_k], weights fp32 [T, top_k]) of logits [T, E]."""
    import torch

    code = _dtype_code(getattr(logits, "dtype", None), "logits")
    stride = _need_rows(logits, "logits")
    (T, E), dev = logits.shape, logits.device
    if bias is not None:
        _need(bias, "bias", torch.float32, E, dev)
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    with _on_gpu(dev):
        nvfp4_route(logits.data_ptr(), code, T, E, top_k, ids.data_ptr(), weights.data_ptr(), score,
                    bias.data_ptr() if bias is not None else 0, groups, top_groups, renormalize, weight_scale,
                    stride, _stream_handle(stream, dev))
    return ids, weights


def moe_sort(ids, E: int, stream=None) -> dict:
    """Sort the choices ids [T, top_k] (int32) by expert: rows [T, top_k], counts [E], starts [E],
    the plan of the products and the capacity and tile of the experts' rows."""
    import torch

    if ids.dim() != 2:
        raise ValueError("ids must be [T, top_k]")
    T, k = ids.shape
    dev = ids.device
    _need(ids, "ids", torch.int32, T * k, dev)
    shape = nvfp4_moe_shape(T, k, E)
    out = {"rows": torch.empty((T, k), dtype=torch.int32, device=dev),
           "counts": torch.empty(E, dtype=torch.int32, device=dev),
           "starts": torch.empty(E, dtype=torch.int32, device=dev),
           "plan": torch.empty(shape["plan_bytes"], dtype=torch.uint8, device=dev),
           "row_capacity": shape["row_capacity"], "tile_rows": shape["tile_rows"], "experts": E}
    with _on_gpu(dev):
        nvfp4_moe_sort(ids.data_ptr(), T, k, E, out["rows"].data_ptr(), out["counts"].data_ptr(),
                       out["starts"].data_ptr(), out["plan"].data_ptr(), _stream_handle(stream, dev))
    return out


def _need_sorted(order, b, sfb, dev):
    import torch

    T, k = order["rows"].shape
    E, rows = order["experts"], order["row_capacity"]
    shape = nvfp4_moe_shape(T, k, E)
    _need(order["plan"], "plan", torch.uint8, shape["plan_bytes"], dev)
    if b.dim() != 2:
        raise ValueError("b must be [row_capacity, K//2]")
    K = 2 * b.shape[1]
    if K % 32:
        raise ValueError(f"b has rows of {K} elements, expected a multiple of 32")
    _need(b, "b", torch.uint8, rows * (K // 2), dev)
    _need(sfb, "sfb", torch.uint8, nvfp4_permuted_scale_bytes(rows, K, 1), dev)
    return T, k, E, rows, K


def _need_experts(a, sfa, alpha, E, K, dev):
    import torch

    if a.dim() != 3 or a.shape[0] != E or 2 * a.shape[2] != K:
        raise ValueError(f"the weights must be [{E}, M, {K // 2}]")
    M = a.shape[1]
    _need(a, "weights", torch.uint8, a.numel(), dev)
    _need(sfa, "weight scales", torch.uint8, nvfp4_permuted_scale_bytes(M, K, E), dev)
    if alpha is not None:
        _need(alpha, "alpha", torch.float32, E, dev)
    return M


def quantize_rows(x, order, encode_scale: float = 1.0, stream=None):
    """Quantise the tokens x [T, K] into the experts' rows of a moe_sort."""
    import torch

    code = _dtype_code(getattr(x, "dtype", None), "x")
    stride = _need_rows(x, "x")
    (T, K), dev, rows = x.shape, x.device, order["row_capacity"]
    k = order["rows"].shape[1]
    if K % 16:
        raise ValueError(f"x has rows of {K} elements, expected a multiple of 16")
    _need(order["rows"], "rows", torch.int32, T * k, dev)
    q = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
    sf = torch.empty(nvfp4_permuted_scale_bytes(rows, K, 1), dtype=torch.uint8, device=dev)
    with _on_gpu(dev):
        nvfp4_quantize(x.data_ptr(), code, T, K, 1, q.data_ptr(), sf.data_ptr(), SF_PERMUTED_128x4, encode_scale,
                       stride, order["rows"].data_ptr(), k, rows, _stream_handle(stream, dev))
    return q, sf


def moe_gemm(a, sfa, b, sfb, order, alpha=None, activation: int = ACT_NONE, dtype=None, stream=None):
    """c [row_capacity, M] = act(alpha[e] * b a[e]^T) for the experts' rows b of a moe_sort."""
    import torch

    dev = a.device
    T, k, E, rows, K = _need_sorted(order, b, sfb, dev)
    M = _need_experts(a, sfa, alpha, E, K, dev)
    dtype = dtype or torch.float16
    code = _dtype_code(dtype, "dtype")
    c = torch.empty((rows, M), dtype=dtype, device=dev)
    with _on_gpu(dev):
        nvfp4_moe_gemm(a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(), order["plan"].data_ptr(), T,
                       k, E, M, K, c.data_ptr(), code, alpha.data_ptr() if alpha is not None else 0, activation,
                       _stream_handle(stream, dev))
    return c


def moe_gated_gemm(a, sfa, b, sfb, order, alpha=None, activation: int = ACT_SILU, encode_scale: float = 1.0,
                   stream=None):
    """(q [row_capacity, F//2], sf) of act(gate) * input, gate and input the even and odd rows of
    a [E, 2F, K//2], for the experts' rows b of a moe_sort."""
    import torch

    dev = a.device
    T, k, E, rows, K = _need_sorted(order, b, sfb, dev)
    M = _need_experts(a, sfa, alpha, E, K, dev)
    if M % 64:
        raise ValueError(f"the weights have {M} rows, expected a multiple of 64")
    F = M // 2
    q = torch.empty((rows, F // 2), dtype=torch.uint8, device=dev)
    sf = torch.empty(nvfp4_permuted_scale_bytes(rows, F, 1), dtype=torch.uint8, device=dev)
    with _on_gpu(dev):
        nvfp4_moe_gated_gemm(a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr(),
                             order["plan"].data_ptr(), T, k, E, F, K, q.data_ptr(), sf.data_ptr(),
                             alpha.data_ptr() if alpha is not None else 0, activation, encode_scale,
                             _stream_handle(stream, dev))
    return q, sf


def moe_combine(y, order, weights, stream=None):
    """out [T, M] = sum_j weights[t, j] * y[rows[t, j]] (y fp16 or bf16)."""
    import torch

    code = _dtype_code(getattr(y, "dtype", None), "y", ("float16", "bfloat16"))
    if y.dim() != 2:
        raise ValueError("y must be [row_capacity, M]")
    T, k = order["rows"].shape
    M, dev = y.shape[1], y.device
    _need(y, "y", y.dtype, order["row_capacity"] * M, dev)
    _need(weights, "weights", torch.float32, T * k, dev)
    out = torch.empty((T, M), dtype=y.dtype, device=dev)
    with _on_gpu(dev):
        nvfp4_moe_combine(y.data_ptr(), code, order["rows"].data_ptr(), weights.data_ptr(), T, k, M,
                          out.data_ptr(), _stream_handle(stream, dev))
    return out


def moe_ffn(x, ids, weights, w1, sf1, w2, sf2, alpha1=None, alpha2=None, encode_x: float = 1.0,
            encode_h: float = 1.0, activation: int = ACT_SILU, out=None, workspace=None, stream=None):
    """The routed feed-forward layer: out [T, D] from x [T, D] (fp16 or bf16), ids and weights
    [T, top_k], w1 [E, 2F, D//2] (gate and input rows interleaved), w2 [E, D, F//2] and their
    permuted scales.  workspace: a uint8 tensor of nvfp4_moe_ffn_workspace_bytes, or None."""
    import torch

    code = _dtype_code(getattr(x, "dtype", None), "x", ("float16", "bfloat16"))
    stride = _need_rows(x, "x")
    (T, D), dev = x.shape, x.device
    if ids.dim() != 2:
        raise ValueError("ids must be [T, top_k]")
    k = ids.shape[1]
    _need(ids, "ids", torch.int32, T * k, dev)
    _need(weights, "weights", torch.float32, T * k, dev)
    if w1.dim() != 3 or w2.dim() != 3 or 2 * w1.shape[2] != D:
        raise ValueError("w1 must be [E, 2F, D//2] and w2 [E, D, F//2]")
    E, F = w1.shape[0], 2 * w2.shape[2]
    if w1.shape[1] != 2 * F or tuple(w2.shape) != (E, D, F // 2) or D % 32 or F % 32:
        raise ValueError("w1 must be [E, 2F, D//2] and w2 [E, D, F//2], D and F multiples of 32")
    _need_experts(w1, sf1, alpha1, E, D, dev)
    _need_experts(w2, sf2, alpha2, E, F, dev)
    if out is None:
        out = torch.empty((T, D), dtype=x.dtype, device=dev)
    _need(out, "out", x.dtype, T * D, dev)
    need = nvfp4_moe_ffn_workspace_bytes(T, k, E, D, F)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError(f"workspace must be {need} contiguous bytes (uint8)")
    if need and workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, expected {dev}")
    with _on_gpu(dev):
        nvfp4_moe_ffn(x.data_ptr(), code, ids.data_ptr(), weights.data_ptr(), w1.data_ptr(), sf1.data_ptr(),
                      w2.data_ptr(), sf2.data_ptr(), T, k, E, D, F, out.data_ptr(), workspace.data_ptr(),
                      workspace.numel(), alpha1.data_ptr() if alpha1 is not None else 0,
                      alpha2.data_ptr() if alpha2 is not None else 0, encode_x, encode_h, activation, stride,
                      _stream_handle(stream, dev))
    return out
