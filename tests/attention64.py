"""Attention on the 4-bit cache in 64 bits on the GPU, for sizes at which numpy takes too long.  Elementary operations on the oracle's values of the cache."""
import numpy as np
import torch

from oracle import attention as oa
from oracle import layer as ol

DEV = torch.device("cuda:0")


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def pages_of(k, v, page, e=(None, None)):
    """Quantised k and v [tokens, H, D], page after page: uint8 [tokens / page, H, page / 16, 2, D / 64, 576]."""
    sides = []
    for x, scale in zip((k, v), e):
        T, H, D = x.shape
        q, sf = ol.quantize(x if scale is None else x * scale[None, :, None])
        at = (T // page, page // 16, 16, H, D // 64)
        rows = [a.reshape(*at, w).transpose(0, 3, 1, 4, 2, 5).reshape(T // page, H, page // 16, D // 64, 16 * w)
                for a, w in ((q, 32), (sf, 4))]
        sides.append(np.concatenate(rows, axis=-1))
    return np.ascontiguousarray(np.stack(sides, axis=3))


class Pool:
    """Pages of a cache, on the GPU, and their values [slots, H, D] in fp64."""

    def __init__(self, cache, page, e=(None, None)):
        self.cache, self.page = gpu(cache), page
        self.e = [None if x is None else gpu(x) for x in e]
        self.k, self.v = (gpu(x if s is None else x / s[:, None]) for x, s in zip(oa.values(cache), e))

    def call(self):
        return dict(cache=self.cache, encode_k=self.e[0], encode_v=self.e[1])


def attend(q, k, v, scale, length, causal=True, window=0):
    """One sequence: q [n, Hq, D] and its k, v [length, Hkv, D], fp64.  A dict of out, lse; mix = sum p |v| / sum p;
    bend = the largest sum |q k| * scale; total = sum p with the largest p 1; seen: tokens.  Rows that see none: 0, -inf."""
    n, Hq, D = q.shape
    G = Hq // k.shape[1]
    j = torch.arange(length - n, length, device=DEV)[:, None]
    t = torch.arange(length, device=DEV)[None]
    sees = t <= j if causal else torch.ones((n, length), dtype=torch.bool, device=DEV)
    if window:
        sees = sees & (t > j - window)
    r = {name: torch.zeros((n, Hq, D), dtype=torch.float64, device=DEV) for name in ("out", "mix")}
    r |= {name: torch.zeros((n, Hq), dtype=torch.float64, device=DEV) for name in ("bend", "total", "gap", "top")}
    r["lse"] = torch.full((n, Hq), -torch.inf, dtype=torch.float64, device=DEV)
    r["seen"] = sees.sum(1)[:, None].double().expand(n, Hq)
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        s = (q[:, h] @ kk.T * scale).masked_fill(~sees, -torch.inf)
        top = s.amax(1, keepdim=True) if length else torch.full((n, 1), -torch.inf, dtype=torch.float64, device=DEV)
        empty = top == -torch.inf
        p = torch.where(empty, 0.0, torch.exp(s - torch.where(empty, 0.0, top)))
        total = p.sum(1, keepdim=True)
        safe = torch.where(empty, 1.0, total)
        r["out"][:, h], r["mix"][:, h] = p @ vv / safe, p @ vv.abs() / safe
        r["lse"][:, h] = torch.where(empty, -torch.inf, top + torch.log(safe))[:, 0]
        r["total"][:, h] = total[:, 0]
        if length:
            r["bend"][:, h] = (q[:, h].abs() @ kk.abs().T * scale).masked_fill(~sees, 0.0).amax(1)
            best = s.topk(min(2, length), 1)
            r["top"][:, h] = best.indices[:, 0].double()
            if length > 1:
                r["gap"][:, h] = best.values[:, 0] - best.values[:, 1]
    return r
