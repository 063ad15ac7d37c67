"""CPU oracle of the layer operators, in 64 bits (numpy): TEST INFRASTRUCTURE ONLY.

The definitions of ``include/nvfp4_gemv.h`` written out directly; shares no code
with the GPU library.  Codes are uint8 arrays, two E2M1 codes a byte, the low
nibble first; scales are E4M3 bytes [..., rows, K//16] unless said otherwise.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_values(q: np.ndarray) -> np.ndarray:
    """[..., K/2] bytes -> [..., K] values."""
    c = np.stack((q & 15, q >> 4), axis=-1).reshape(*q.shape[:-1], -1)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def e4m3_values(b: np.ndarray) -> np.ndarray:
    e, m = (b.astype(int) >> 3) & 15, b.astype(int) & 7
    v = np.where(e == 0, m / 512.0, (1 + m / 8.0) * np.exp2(e - 7.0))
    v = np.where((b & 0x7F) == 0x7F, np.nan, v)
    return np.where(b & 0x80, -v, v)


def matrix(q: np.ndarray, sf: np.ndarray) -> np.ndarray:
    """The values of a quantised matrix; sf [..., rows, K/16]."""
    return e2m1_values(q) * np.repeat(e4m3_values(sf), 16, axis=-1)


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Bytes of non-negative finite values, to nearest even, at most 448."""
    v = np.minimum(np.asarray(v, dtype=np.float64), 448.0)
    _, e = np.frexp(v)
    e = np.maximum(e - 1, -6)  # exponent of the binade, not below the subnormals'
    n = np.rint(v / np.exp2(e - 3.0))  # units of the last place, half to even
    # n == 16 is the next binade's 8: both give the same byte
    return np.where(v < 2.0 ** -6, n, (e + 7) * 8 + (n - 8)).astype(np.uint8)


def round_e2m1(r: np.ndarray) -> np.ndarray:
    """Codes 0..7 of non-negative values, to nearest even, at most 6."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    code = np.zeros(r.shape, dtype=np.uint8)
    for i, mid in enumerate(mids):  # a tie between codes i and i + 1 goes to the even one
        code += ((r > mid) | ((r == mid) & (i % 2 == 1))).astype(np.uint8)
    return code


def quantize(x: np.ndarray, encode: float = 1.0):
    """(bytes [..., K/2], scales [..., K/16]) of fp32 (or narrower) x."""
    with np.errstate(over="ignore", invalid="ignore"):
        y = (x.astype(np.float32) * np.float32(encode)).astype(np.float64)
    return quantize_values(y)


def quantize_values(y: np.ndarray):
    y = y.reshape(*y.shape[:-1], -1, 16)
    bad = ~np.isfinite(y).all(axis=-1)
    y = np.where(bad[..., None], 0.0, y)
    sf = round_e4m3(np.abs(y).max(axis=-1) / 6.0)
    s = e4m3_values(sf)[..., None]
    r = np.abs(y) / np.where(s > 0, s, np.inf)
    code = round_e2m1(r) | np.where(np.signbit(y) & (s > 0), 8, 0).astype(np.uint8)
    code = code.reshape(*code.shape[:-2], -1)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), np.where(bad, 0x7F, sf).astype(np.uint8)


def atoms(sf: np.ndarray) -> np.ndarray:
    """Scales [L, rows, K/16] -> flat 128x4 atoms, zero padding."""
    L, rows, kb = sf.shape
    rm, rk = -(-rows // 128), -(-kb // 4)
    full = np.zeros((L, rm * 128, rk * 4), dtype=np.uint8)
    full[:, :rows, :kb] = sf
    return full.reshape(L, rm, 4, 32, rk, 4).transpose(0, 1, 4, 3, 2, 5).reshape(-1).copy()


def from_atoms(flat: np.ndarray, rows: int, kb: int, L: int = 1) -> np.ndarray:
    rm, rk = -(-rows // 128), -(-kb // 4)
    full = flat.reshape(L, rm, rk, 32, 4, 4).transpose(0, 1, 4, 3, 2, 5).reshape(L, rm * 128, rk * 4)
    return full[:, :rows, :kb].copy()


def activation(y: np.ndarray, act: int) -> np.ndarray:
    from math import erf, sqrt

    with np.errstate(over="ignore", invalid="ignore"):
        if act == 1:
            return np.where(np.isnan(y), y, np.maximum(y, 0.0))
        if act == 2:
            return y / (1 + np.exp(-y))
        if act == 3:
            return 0.5 * y * (1 + np.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))
        if act == 4:
            return 0.5 * y * (1 + np.vectorize(erf)(y / sqrt(2)))
    return y


def gemm(a: np.ndarray, b: np.ndarray, alpha: float = 1.0, bias=None, act: int = 0):
    """(c [L, N, M], sum of |terms| times |alpha|) of value matrices a [L, M, K], b [L, N, K]."""
    c = np.einsum("lnk,lmk->lnm", b, a) * alpha
    if bias is not None:
        c = c + bias[:, None, :]
    return activation(c, act), np.einsum("lnk,lmk->lnm", np.abs(b), np.abs(a)) * abs(alpha)


def route(logits, top_k, sigmoid=False, bias=None, groups=1, top_groups=1, renormalize=True, scale=1.0):
    """(ids, weights, ranks): ranks [T, E] with masked experts at -inf."""
    x = np.where(np.isnan(logits), -np.inf, logits.astype(np.float64))
    T, E = x.shape
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        if sigmoid:
            score = 1 / (1 + np.exp(-x))
        else:
            top = x.max(axis=1, keepdims=True)
            e = np.where(x == top, np.where(top == -np.inf, 0.0, 1.0), np.exp(x - top))
            total = e.sum(axis=1, keepdims=True)
            score = np.where(total > 0, e / np.where(total > 0, total, 1), 0.0)
        biased = score if bias is None else score + bias.astype(np.float64)
        rank = x if bias is None else np.where(x == -np.inf, -np.inf, biased)
        rank = np.where(np.isnan(rank), -np.inf, rank)
    open_ = np.ones((T, E), dtype=bool)
    if groups > 1:
        per = E // groups
        best = np.sort(np.where(rank == -np.inf, -np.inf, biased).reshape(T, groups, per), axis=2)[:, :, ::-1]
        two = best[:, :, :2]
        gscore = np.where(two[:, :, 0] == -np.inf, -np.inf, np.where(two == -np.inf, 0.0, two).sum(axis=2))
        order = np.argsort(-gscore, axis=1, kind="stable")[:, :top_groups]
        keep = np.zeros((T, groups), dtype=bool)
        np.put_along_axis(keep, order, True, axis=1)
        open_ = np.repeat(keep, per, axis=1)
    rank = np.where(open_, rank, -np.inf)
    ids = np.argsort(-rank, axis=1, kind="stable")[:, :top_k]
    chosen = np.take_along_axis(rank, ids, axis=1) > -np.inf
    w = np.where(chosen, np.take_along_axis(score, ids, axis=1), 0.0)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)
    return np.where(chosen, ids, -1), w * scale, rank


def moe_rows(ids: np.ndarray, E: int, tile_rows: int):
    """(rows [T, k], counts [E], starts [E]) of the stable sort by expert."""
    pitch = max(tile_rows, 128)
    flat = ids.reshape(-1)
    rows = np.full(flat.shape, -1, dtype=np.int64)
    counts = np.array([(flat == e).sum() for e in range(E)])
    tiles = -(-counts // tile_rows)
    first = np.concatenate(([0], np.cumsum(tiles)[:-1]))
    for e in range(E):
        at = np.nonzero(flat == e)[0]
        rank = np.arange(at.size)
        rows[at] = (first[e] + rank // tile_rows) * pitch + rank % tile_rows
    return rows.reshape(ids.shape), counts, first * pitch
