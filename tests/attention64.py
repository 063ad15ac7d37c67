"""Attention on the 4-bit cache in 64 bits on the GPU, for sizes at which numpy takes too long, and what the
kernels' arithmetic may be off by.  Elementary operations on the oracle's values of the cache."""
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


def bounds(r, D, half, largest, run):
    """Of (out, lse): `half` the half step of out's type, `largest` the largest |v|, `run` the tokens that one
    thread's sums go over before they are added to others' (those of some 16 warps and 152 CTAs, at most).

    A score is an fp32 sum of D products, in D/16 steps that may each lose 2^-22 of what is summed, and four more
    roundings of its size: d = (D/16 + 4) 2^-22 bend.  A p is off by 2 d (its own score and the maximum's) and by the
    exponential's 2^-22; in the product with v, where it is fp16 with the reference at 2^7, by 2^-11 of itself or by
    2^-25 2^-7 of the largest p.  Sums of p: run/4 additions of a thread at most (a lane of eight takes 1/8 of the
    tokens, a row's four partial sums 1/4 each) and 168 more, 2^-24 each.  Sums of p v: run/16 steps and as many
    rescalings at most, 2^-22 each, and the 168."""
    d = r["bend"] * (D / 16 + 4) * 2.0 ** -22
    sums, steps = (run / 4 + 168) * 2.0 ** -24, (run / 16 + 64) * 2.0 ** -22
    p = 2 * d + 2.0 ** -22
    small = r["seen"] * 2.0 ** -32 * largest / r["total"].clamp(min=1.0)
    wide = (2 * p + 2.0 ** -11 + sums + steps)[..., None] * r["mix"] + small[..., None] + half * r["out"].abs()
    # (second-order terms; the smallest numbers of the types)
    return wide * (1 + 2.0 ** -6) + 2.0 ** -24, (2 * p + sums) * (1 + 2.0 ** -6) + 2.0 ** -22 + 2.0 ** -22 * r["bend"]


def check(pool, q, table, lens, counts, out, lse, run, scale=None, causal=True, window=0):
    """A call's results against the definition, sequence by sequence; table and lens as numpy arrays."""
    D, half = q.shape[2], torch.finfo(out.dtype).eps / 2
    at = 0
    for b, (length, n) in enumerate(zip(lens, counts)):
        length, n = int(length), int(n)
        if n == 0:
            continue
        t = np.arange(length)
        slots = gpu(table[b, t // pool.page].astype(np.int64) * pool.page + t % pool.page)
        r = attend(q[at: at + n].double(), pool.k[slots], pool.v[slots], scale or D ** -0.5, length, causal, window)
        tol, tol_lse = bounds(r, D, half, pool.v.abs().max(), run if isinstance(run, (int, float)) else run[b])
        got, got_lse = out[at: at + n].double(), lse[at: at + n].double()
        assert not got.isnan().any(), b
        worst = ((got - r["out"]).abs() - tol).max().item()
        assert worst <= 0, (b, length, n, worst)
        empty = r["lse"] == -torch.inf
        assert (got_lse[empty] == -torch.inf).all() and not got[empty].any(), b
        off = ((got_lse - r["lse"]).abs() - tol_lse)[~empty]
        assert not empty.logical_not().any() or off.max().item() <= 0, (b, length, n, off.max().item())
        at += n
