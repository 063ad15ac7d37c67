"""The operators of attention: rotary positions, the 4-bit key and value cache, attention on it.

The same thin binding as the layer operators' (``layer.py``): ``nvfp4_*`` functions take
device pointers as integers, the functions without the prefix take torch tensors, check them
and allocate the outputs.  ``include/nvfp4_gemv.h`` defines each call; ``rope_table`` is host
arithmetic on a few dozen numbers, for the program to call once.

There are no gradients, as in the layer operators, but for the rotation's own: the gradient of
``rope(x, ...)`` is ``rope(grad, ..., inverse=True)``.
"""
from __future__ import annotations

import ctypes
import math

from . import _check, library
from . import layer as _layer
from .layer import _dtype_code, _empty, _enqueue, _load, _ptr

GRANULE_TOKENS = 16
MOST = (1 << 31) - 1  # the largest number of an option; no sequence has as many tokens
LEAST_SCALE = 2.0 ** -149  # fp32's smallest number; what rounds to 0 would be taken for the default
PLANE_BYTES = 576  # 16 tokens x 64 elements: 32 bytes of codes and 4 of scales a token


class _RopeOptions(ctypes.Structure):
    _fields_ = [("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32), ("factor", ctypes.c_float),
                ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64)]


class _KvRows(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("encode_k", ctypes.c_void_p),
                ("encode_v", ctypes.c_void_p), ("k_token_stride", ctypes.c_int64),
                ("k_head_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64),
                ("v_head_stride", ctypes.c_int64)]


class _AttentionOptions(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("q_starts", ctypes.c_void_p), ("encode_k", ctypes.c_void_p),
                ("encode_v", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64)]


def declare(lib: ctypes.CDLL) -> None:
    """Argument types of the attention calls."""
    P, I64, I, Z = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    R = ctypes.POINTER
    for name, args, result in (
            ("nvfp4_rope", [P, I, I64, I64, I64, P, P, I64, R(_RopeOptions), P, P], I),
            ("nvfp4_kv_cache_bytes", [I64] * 4, Z),
            ("nvfp4_kv_write", [R(_KvRows), I, I64, I64, I64, P, P, I64, I64, P], I),
            ("nvfp4_kv_read", [R(_KvRows), I, I64, I64, I64, P, P, I64, I64, P], I),
            ("nvfp4_attention_workspace_bytes", [I64] * 7 + [I, I64], Z),
            ("nvfp4_attention", [P, I, I64, I64, I64, I64, P, I64, I64, P, I64, P, I64, R(_AttentionOptions), P, P, Z,
                                 P], I)):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = result


def _limit(name: str, value: int) -> int:
    """A limit on tokens, for a field of 32 bits (which would take others modulo 2^32)."""
    if value < 0:
        raise ValueError(f"{name} is {value}, expected 0 or more")
    return value if value < MOST else MOST


# ---------------------------------------------------------------------------
# device pointers
# ---------------------------------------------------------------------------

def nvfp4_rope(x: int, dtype: int, T: int, H: int, D: int, positions: int, table: int, pairs: int, y: int,
               interleaved: bool = False, inverse: bool = False, factor: float = 1.0, x_token_stride: int = 0,
               x_head_stride: int = 0, y_token_stride: int = 0, y_head_stride: int = 0, stream: int = 0) -> None:
    """Enqueue the rotation of x [T][H][D] into y."""
    opt = _RopeOptions(1 if interleaved else 0, 1 if inverse else 0, factor, x_token_stride, x_head_stride,
                       y_token_stride, y_head_stride)
    _check(library().nvfp4_rope(x, dtype, T, H, D, positions, table, pairs, ctypes.byref(opt), y, stream),
           "nvfp4_rope")


def nvfp4_kv_cache_bytes(pages: int, heads: int, D: int, page_size: int) -> int:
    return int(library().nvfp4_kv_cache_bytes(pages, heads, D, page_size))


def nvfp4_kv_write(k: int, v: int, dtype: int, T: int, heads: int, D: int, slots: int, cache: int, pages: int,
                   page_size: int, encode_k: int = 0, encode_v: int = 0, strides=(0, 0, 0, 0),
                   stream: int = 0) -> None:
    """Enqueue the quantisation of k and v [T][heads][D] into their slots; strides are k's token
    and head strides, then v's."""
    rows = _KvRows(k or None, v or None, encode_k or None, encode_v or None, *strides)
    _check(library().nvfp4_kv_write(ctypes.byref(rows), dtype, T, heads, D, slots, cache, pages, page_size, stream),
           "nvfp4_kv_write")


def nvfp4_kv_read(k: int, v: int, dtype: int, T: int, heads: int, D: int, slots: int, cache: int, pages: int,
                  page_size: int, encode_k: int = 0, encode_v: int = 0, strides=(0, 0, 0, 0),
                  stream: int = 0) -> None:
    """Enqueue k and v [T][heads][D] (0: not wanted) = the values of their slots."""
    rows = _KvRows(k or None, v or None, encode_k or None, encode_v or None, *strides)
    _check(library().nvfp4_kv_read(ctypes.byref(rows), dtype, T, heads, D, slots, cache, pages, page_size, stream),
           "nvfp4_kv_read")


def nvfp4_attention_workspace_bytes(T: int, B: int, Hq: int, Hkv: int, D: int, page_size: int, max_pages: int,
                                    ragged: bool = False, max_q: int = 0) -> int:
    return int(library().nvfp4_attention_workspace_bytes(T, B, Hq, Hkv, D, page_size, max_pages, 1 if ragged else 0,
                                                         max_q))


def nvfp4_attention(q: int, dtype: int, T: int, Hq: int, Hkv: int, D: int, cache: int, pages: int, page_size: int,
                    page_table: int, max_pages: int, lengths: int, B: int, out: int, workspace: int,
                    workspace_bytes: int, scale: float = 0.0, causal: bool = True, window: int = 0, max_q: int = 0,
                    q_starts: int = 0, encode_k: int = 0, encode_v: int = 0, lse: int = 0, q_token_stride: int = 0,
                    q_head_stride: int = 0, stream: int = 0) -> None:
    """Enqueue the attention of q [T][Hq][D] on the cache."""
    opt = _AttentionOptions(LEAST_SCALE if 0 < scale < LEAST_SCALE else scale, 1 if causal else 0,
                            _limit("window", window), _limit("max_q", max_q),
                            q_starts or None, encode_k or None,
                            encode_v or None, lse or None, q_token_stride, q_head_stride)
    _check(library().nvfp4_attention(q, dtype, T, Hq, Hkv, D, cache, pages, page_size, page_table, max_pages, lengths,
                                     B, ctypes.byref(opt), out, workspace, workspace_bytes, stream),
           "nvfp4_attention")


# ---------------------------------------------------------------------------
# torch tensors
# ---------------------------------------------------------------------------

def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original: int = 0, low: float = 1.0, high: float = 32.0) -> list:
    """Radians per position of each pair of a rotated head, base ** (-2 i / rotary_dim), for
    contexts `factor` times the `original` length:

    none     as they are
    linear   all divided by factor
    base     of a base that grows by factor ** (rotary_dim / (rotary_dim - 2))
    ramp     pairs that turn more than `high` times within the original length stay, those that turn
             less than `low` times are divided by factor, and between them a ramp over the pairs' index
    bands    the same with the ramp over the turns within the original length
    """
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim is {rotary_dim}, expected an even number of elements")
    if scaling not in ("none", "linear", "base", "ramp", "bands"):
        raise ValueError(f"scaling is {scaling!r}, expected none, linear, base, ramp or bands")
    if not base > 1 or not factor > 0 or not math.isfinite(base) or not math.isfinite(factor):
        raise ValueError("base must be above 1 and factor above 0")
    if scaling in ("ramp", "bands") and not (original > 0 and 0 < low < high):
        raise ValueError(f"{scaling} needs the original length and 0 < low < high")
    if scaling == "base":
        if rotary_dim == 2:
            raise ValueError("a single pair has no base to scale")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    out = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling == "linear":
        out = [f / factor for f in out]
    elif scaling == "ramp":
        first, last = (rotary_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
                       for turns in (high, low))
        first, last = max(math.floor(first), 0), min(math.ceil(last), rotary_dim - 1)
        for i, f in enumerate(out):
            part = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            out[i] = f / factor * part + f * (1 - part)
    elif scaling == "bands":
        for i, f in enumerate(out):
            part = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            out[i] = f * part + f / factor * (1 - part)
    return out


def rope_table(rotary_dim: int = 0, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original: int = 0, low: float = 1.0, high: float = 32.0, frequencies=None, device="cuda"):
    """The table of rope(): int64 [pairs] in 2^-64 turns per position, from rope_frequencies() or
    from `frequencies` (radians per position).  Made once, on the host."""
    torch = _load()
    if frequencies is None:
        frequencies = rope_frequencies(rotary_dim, base, scaling, factor, original, low, high)
    rows = []
    for f in frequencies:
        if not math.isfinite(f):
            raise ValueError(f"a frequency is {f}")
        turns = round(math.ldexp(f / (2 * math.pi), 64)) % (1 << 64)
        rows.append(turns - (1 << 64) if turns >> 63 else turns)
    if not rows:
        raise ValueError("there are no frequencies")
    return torch.tensor(rows, dtype=torch.int64, device=device)


def _heads(x, name, device=None):
    """[T, H, D] with contiguous heads: T, H, D, token stride, head stride (dense ones where nothing steps by them)."""
    shape, stride = x.shape, x.stride()
    if len(shape) == 3 and stride[2] == 1 and stride[1] >= shape[2] and \
            stride[0] >= (shape[1] - 1) * stride[1] + shape[2] and (device is None or x.device == device):
        # (the usual case in few steps)
        T, H, D = shape
        head = stride[1] if H > 1 else D
        return T, H, D, stride[0] if T > 1 else H * head, head
    if x.dim() != 3:
        raise ValueError(f"{name} must be [T, H, D]")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, expected {device}")
    T, H, D = x.shape
    token, head, step = x.stride()
    if D > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous heads")
    if H <= 1:
        head = D
    if T <= 1:
        token = H * head
    # heads of a token beside each other, or tokens of a head
    if T * H * D and ((H > 1 and head < D) or (T > 1 and token < D) or (
            T > 1 and H > 1 and token < (H - 1) * head + D and head < (T - 1) * token + D)):
        raise ValueError(f"{name} must have heads that do not overlap")
    return T, H, D, token, head


def rope(x, positions, table, interleaved: bool = False, factor: float = 1.0, inverse: bool = False, out=None,
         stream=None):
    """x [T, H, D] (fp16, bf16 or fp32, heads contiguous) with the first 2 * len(table) elements of
    every head turned by positions [T] (int32) times the table's frequencies, in pairs (i, pairs + i) or,
    interleaved, (2i, 2i + 1), and multiplied by factor.  inverse turns back, which is the gradient.
    out: x itself (in place), or a tensor that does not overlap it."""
    torch = _layer._torch or _load()
    code = _dtype_code(x, "x")
    T, H, D, token, head = _heads(x, "x")
    dev, pairs = x.device, table.numel()
    if not 1 <= pairs <= D // 2:
        raise ValueError(f"the table has {pairs} pairs, heads have {D} elements")
    pp, tp = _ptr(positions, "positions", torch.int32, T, dev), _ptr(table, "table", torch.int64, pairs, dev)
    if out is None:
        out = _empty((T, H, D), x.dtype, dev, stream)
        y_token, y_head = H * D, D
    else:
        if out.shape != x.shape or out.dtype is not x.dtype:
            raise ValueError("out must have the shape and type of x")
        _, _, _, y_token, y_head = _heads(out, "out", dev)
        if T * H * D and out.data_ptr() != x.data_ptr():
            a, b = x.data_ptr(), out.data_ptr()
            size = x.element_size()
            if a < b + ((T - 1) * y_token + (H - 1) * y_head + D) * size and \
                    b < a + ((T - 1) * token + (H - 1) * head + D) * size and \
                    not _apart(a, b, (token, head), (y_token, y_head), H, D, size):
                raise ValueError("out must be x or not overlap it")
    _enqueue("nvfp4_rope", dev, stream, x.data_ptr(), code, T, H, D, pp, tp, pairs,
             ctypes.byref(_RopeOptions(1 if interleaved else 0, 1 if inverse else 0, factor, token, head, y_token,
                                       y_head)), out.data_ptr())
    return out


def _apart(a, b, x_strides, y_strides, H, D, size) -> bool:
    """Whether two views of the same rows (a fused buffer) share no element: equal strides, and
    heads that lie beside each other within a token."""
    if x_strides != y_strides or (b - a) % size:
        return False
    token, head = x_strides
    width = (H - 1) * head + D
    gap = (b - a) // size % token if token else 0
    return width <= gap <= token - width


def _torch():
    return _layer._torch or _load()


def kv_cache(pages: int, heads: int, head_dim: int, page_size: int = 64, device="cuda"):
    """An empty cache: uint8 [pages, heads, page_size / 16, 2, head_dim / 64, 576] (see nvfp4_kv_write)."""
    torch = _torch()
    _check_sizes(heads, head_dim, page_size)
    if pages < 0:
        raise ValueError(f"pages is {pages}")
    return torch.zeros((pages, heads, page_size // GRANULE_TOKENS, 2, head_dim // 64, PLANE_BYTES),
                       dtype=torch.uint8, device=device)


def _check_sizes(heads, head_dim, page_size):
    if head_dim not in (64, 128, 256):
        raise ValueError(f"head_dim is {head_dim}, expected 64, 128 or 256")
    if page_size < 16 or page_size % 16:
        raise ValueError(f"page_size is {page_size}, expected a multiple of 16")
    if heads < 1:
        raise ValueError(f"heads is {heads}")


def _cache(cache, device):
    """(address, pages, heads, head_dim, page_size) of a cache."""
    torch = _torch()
    shape = cache.shape
    if len(shape) != 6 or shape[3] != 2 or shape[5] != PLANE_BYTES or shape[4] not in (1, 2, 4):
        raise ValueError("cache must be [pages, heads, page_size / 16, 2, head_dim / 64, 576], head_dim 64, 128 or 256")
    pages, heads, granules, _, planes, _ = shape
    return (_ptr(cache, "cache", torch.uint8, cache.numel(), device), pages, heads, planes * 64,
            granules * GRANULE_TOKENS)


def _encode(t, name, heads, device):
    return None if t is None else _ptr(t, name, _torch().float32, heads, device)


def kv_write(k, v, cache, slots, encode_k=None, encode_v=None, stream=None):
    """Quantise k and v [T, heads, D] (fp16, bf16 or fp32, heads contiguous), times the encode scales
    (fp32 [heads]), into the slots (int64 [T], page * page_size + place) of a kv_cache(); a slot outside
    the cache (-1) is skipped, none may be named twice.  Returns the cache."""
    torch = _torch()
    code, dev = _dtype_code(k, "k"), k.device
    T, H, D, k_token, k_head = _heads(k, "k")
    if v.shape != k.shape or v.dtype is not k.dtype:
        raise ValueError("v must have the shape and type of k")
    _, _, _, v_token, v_head = _heads(v, "v", dev)
    cp, pages, heads, head_dim, page = _cache(cache, dev)
    if (H, D) != (heads, head_dim):
        raise ValueError(f"k has {H} heads of {D}, the cache {heads} of {head_dim}")
    rows = _KvRows(k.data_ptr(), v.data_ptr(), _encode(encode_k, "encode_k", H, dev),
                   _encode(encode_v, "encode_v", H, dev), k_token, k_head, v_token, v_head)
    _enqueue("nvfp4_kv_write", dev, stream, ctypes.byref(rows), code, T, H, D,
             _ptr(slots, "slots", torch.int64, T, dev), cp, pages, page)
    return cache


def kv_read(cache, slots, dtype=None, encode_k=None, encode_v=None, stream=None):
    """(k, v) [T, heads, D] of the slots (int64 [T]) of a cache, as dtype (default float32): code * scale
    / encode; zeros for slots outside the cache."""
    torch = _torch()
    dtype = dtype or torch.float32
    code, dev = _dtype_code(dtype, "dtype"), cache.device
    cp, pages, H, D, page = _cache(cache, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be [T]")
    T = slots.numel()
    sp = _ptr(slots, "slots", torch.int64, T, dev)
    k, v = _empty((T, H, D), dtype, dev, stream), _empty((T, H, D), dtype, dev, stream)
    rows = _KvRows(k.data_ptr(), v.data_ptr(), _encode(encode_k, "encode_k", H, dev),
                   _encode(encode_v, "encode_v", H, dev), 0, 0, 0, 0)
    _enqueue("nvfp4_kv_read", dev, stream, ctypes.byref(rows), code, T, H, D, sp, cp, pages, page)
    return k, v


_workspaces = {}  # workspace bytes of sizes


def attention(q, cache, page_table, lengths, q_starts=None, max_q: int = 0, scale: float = 0.0, causal: bool = True,
              window: int = 0, encode_k=None, encode_v=None, return_lse: bool = False, out=None, workspace=None,
              stream=None):
    """out [T, Hq, D] of q [T, Hq, D] (fp16 or bf16, heads contiguous) on a kv_cache().

    page_table int32 [B, max_pages] and lengths int32 [B] (contiguous) say what each sequence has cached, its query
    tokens (T / B each, or rows q_starts[b] to q_starts[b + 1] - 1, at most max_q, or 0: any number) among
    them as its last ones.  A query sees the tokens up to its own (causal), the last `window` of them, or all.  scale 0 is
    1 / sqrt(D).  return_lse: (out, lse fp32 [T, Hq]).  workspace: a uint8 tensor of
    nvfp4_attention_workspace_bytes, or None; calls that may run at once need one each."""
    torch = _torch()
    code, dev = _dtype_code(q, "q", fp32=False), q.device
    T, Hq, D, token, head = _heads(q, "q")
    cp, pages, Hkv, head_dim, page = _cache(cache, dev)
    if D != head_dim or Hq % Hkv or Hq == 0:
        raise ValueError(f"q has {Hq} heads of {D}, the cache {Hkv} of {head_dim}")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    i32 = torch.int32
    tp, lp = _ptr(page_table, "page_table", i32, B * max_pages, dev), _ptr(lengths, "lengths", i32, B, dev)
    if q_starts is None:
        if T % B if B else T:
            raise ValueError(f"q has {T} tokens for {B} sequences")
        starts, max_q = None, 0
    else:
        starts, max_q = _ptr(q_starts, "q_starts", i32, B + 1, dev), min(_limit("max_q", max_q), T)
    if token % 8 or head % 8 or q.data_ptr() % 16:
        raise ValueError("q must have 16-byte aligned heads")
    if out is None:
        # rows that belong to no sequence are not written
        out = _empty((T, Hq, D), q.dtype, dev, stream)
    else:
        a, b, size = q.data_ptr(), _ptr(out, "out", q.dtype, T * Hq * D, dev), 2
        if T and a < b + T * Hq * D * size and b < a + ((T - 1) * token + (Hq - 1) * head + D) * size:
            raise ValueError("out must not overlap q")
    lse = _empty((T, Hq), torch.float32, dev, stream) if return_lse else None
    sizes = (T, B, Hq, Hkv, D, page, max_pages, 0 if starts is None else 1, max_q)
    need = _workspaces.get(sizes)
    if need is None:
        if len(_workspaces) > 4096:
            _workspaces.clear()
        need = _workspaces[sizes] = library().nvfp4_attention_workspace_bytes(*sizes)
    if workspace is None:
        workspace, size = _empty(need, torch.uint8, dev, stream), need
    else:
        size = workspace.numel()
        if size < need:
            raise ValueError(f"workspace has {size} bytes, expected {need}")
        _ptr(workspace, "workspace", torch.uint8, size, dev)
    if 0 < scale < LEAST_SCALE:
        scale = LEAST_SCALE
    opt = _AttentionOptions(scale, 1 if causal else 0, _limit("window", window), max_q, starts, _encode(encode_k, "encode_k", Hkv, dev),
                            _encode(encode_v, "encode_v", Hkv, dev), None if lse is None else lse.data_ptr(), token,
                            head)
    _enqueue("nvfp4_attention", dev, stream, q.data_ptr(), code, T, Hq, Hkv, D, cp, pages, page, tp, max_pages, lp, B,
             ctypes.byref(opt), out.data_ptr(), workspace.data_ptr(), size)
    return (out, lse) if return_lse else out
