"""CPU oracle of the operators of attention, in 64 bits (numpy): TEST INFRASTRUCTURE ONLY.

The definitions of ``include/nvfp4_gemv.h`` written out directly; shares no code with the GPU
library.
"""
from __future__ import annotations

import numpy as np

from . import layer as ol


def turns(positions, table):
    """[T, pairs] fractions of a turn, exactly (position * f modulo 2^64, in whole numbers)."""
    return np.array([[((int(p) * int(f)) % (1 << 64)) / 2.0 ** 64 for f in table] for p in positions])


def rope(x, positions, table, interleaved=False, factor=1.0, inverse=False):
    """x [T, H, D] values."""
    a = 2 * np.pi * turns(positions, table)[:, None, :] * (-1 if inverse else 1)
    n = len(table)
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    y = x.astype(np.float64).copy()
    u, w = y[..., first], y[..., second]
    y[..., first] = (u * np.cos(a) - w * np.sin(a)) * factor
    y[..., second] = (w * np.cos(a) + u * np.sin(a)) * factor
    return y


def empty_cache(pages, heads, D, page_size, fill=0):
    return np.full((pages, heads, page_size // 16, 2, D // 64, 576), fill, dtype=np.uint8)


def write(cache, slots, k, v, encode_k=None, encode_v=None):
    """Quantise k and v [T, heads, D] (fp32 or narrower) into the slots, one byte after the other."""
    pages, heads, granules, _, planes, _ = cache.shape
    for side, (x, e) in enumerate(((k, encode_k), (v, encode_v))):
        for t, slot in enumerate(slots):
            if not 0 <= slot < pages * granules * 16:
                continue
            page, at = divmod(int(slot), granules * 16)
            for h in range(heads):
                q, sf = ol.quantize(x[t, h][None], 1.0 if e is None else e[h])
                for c in range(planes):
                    plane = cache[page, h, at // 16, side, c]
                    plane[at % 16 * 32: at % 16 * 32 + 32] = q[0, c * 32: c * 32 + 32]
                    plane[512 + at % 16 * 4: 512 + at % 16 * 4 + 4] = sf[0, c * 4: c * 4 + 4]


def values(cache):
    """(k, v) [pages * page_size, heads, D] values of all slots."""
    pages, heads, granules, _, planes, _ = cache.shape
    q = cache[..., :512].reshape(pages, heads, granules, 2, planes, 16, 32)
    s = cache[..., 512:].reshape(pages, heads, granules, 2, planes, 16, 4)
    x = ol.matrix(q, s)  # [..., 16, 64]
    x = x.transpose(3, 0, 2, 5, 1, 4, 6).reshape(2, pages * granules * 16, heads, planes * 64)
    return x[0], x[1]


def attention(q, k, v, scale, length, causal=True, window=0):
    """One sequence: q [n, Hq, D], k and v [>= length, Hkv, D] values, decoded.  Returns (out, lse, mix,
    bend): mix is sum p |v| / sum p, what the rounding of p acts on, and bend sum |q k| * scale of a
    row's worst token, what the rounding of a score acts on.  Rows without a token: 0 and -inf."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    out, mix = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse, bend = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        j = length - n + i
        hi = j + 1 if causal else length
        lo = max(0, j + 1 - window) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            kk, vv = k[lo:hi, h * Hkv // Hq], v[lo:hi, h * Hkv // Hq]
            s = kk @ q[i, h] * scale
            bend[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
            p = np.exp(s - s.max())
            out[i, h], mix[i, h] = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
            lse[i, h] = s.max() + np.log(p.sum())
    return out, lse, mix, bend


def tolerance(out, mix, bend, length, D, eps, largest):
    """Bounds of (out, lse) for the kernels' arithmetic: eps the half step of out's type, largest the
    largest |v|.

    A score is an fp32 sum of D products, in D/16 steps that may each lose 2^-22 of what is summed, and
    two more roundings: d = (D/16 + 4) 2^-22 bend.  A p is off by 2 d (its own and the maximum's score),
    by the exponential's 2^-22 and, in the product, by fp16's half step: 2^-11, or 2^-25 of the largest p
    where it is below 2^-14 of that.  The sums over length tokens, of p and of p v, have length/16 + 64
    steps of 2^-22 each.  So out is off by mix times these, by length 2^-25 largest for the smallest
    p, and by eps of itself."""
    d = bend * (D / 16 + 4) * 2.0 ** -22
    steps = (length / 16 + 64) * 2.0 ** -22
    rel = 2 * d + 2.0 ** -22 + 2.0 ** -11 + 2 * steps
    # (the last factors: second-order terms, and fp16's and bf16's smallest numbers)
    wide = (rel[..., None] * mix + length * 2.0 ** -25 * largest + eps * np.abs(out)) * (1 + 2.0 ** -6) + 2.0 ** -24
    return wide, 2 * d + 2.0 ** -21 + 2 * steps + 2.0 ** -22 * np.abs(bend)
