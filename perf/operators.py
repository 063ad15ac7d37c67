"""The NVFP4 layer operators, as a program that serves a model calls them.

Four operators around the block-scaled product, each with its plain form:

  quantize  16-bit or 32-bit rows -> E2M1 codes and E4M3 block scales, and back
  gemm      quantised rows times quantised weights, any number of rows
  route     scores of the experts -> each token's experts and their weights
  experts   the routed, gated feed-forward layer on NVFP4 experts

``own`` chooses between the plain form (elementary torch operations in fp32)
and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # one token's hidden state before a projection: launch latency
        dict(name="quantize_1x4096_bf16", op="quantize", rows=1, K=4096, dtype="bf16", layout="permuted",
             encode=1.0, pad=0),
        # a ragged prompt, rows of a wider buffer, plain scales, a per-tensor scale
        dict(name="quantize_777x7168_fp16_plain", op="quantize", rows=777, K=7168, dtype="fp16",
             layout="plain", encode=3.7, pad=64),
        # a full batch of prompts
        dict(name="quantize_16384x8192_bf16", op="quantize", rows=16384, K=8192, dtype="bf16",
             layout="permuted", encode=0.81, pad=0),
        # a decode batch beyond 16 tokens
        dict(name="gemm_24x7168x2048_bf16", op="gemm", N=24, M=7168, K=2048, L=1, dtype="bf16",
             bias=False, act="none"),
        # odd sizes everywhere, two batches, the epilogue in use
        dict(name="gemm_333x5000x4128_fp16_gelu", op="gemm", N=333, M=5000, K=4128, L=2, dtype="fp16",
             bias=True, act="gelu_tanh"),
        # a long prompt through a square projection
        dict(name="gemm_8192x8192x8192_bf16", op="gemm", N=8192, M=8192, K=8192, L=1, dtype="bf16",
             bias=False, act="none"),
        # one token among few experts
        dict(name="route_1x64_softmax_top6", op="route", T=1, E=64, k=6, dtype="fp32", score="softmax",
             bias=False, groups=1, top_groups=1),
        # 16-bit scores, many ties, an expert count that is no power of two
        dict(name="route_1111x160_softmax_top6_bf16", op="route", T=1111, E=160, k=6, dtype="bf16",
             score="softmax", bias=False, groups=1, top_groups=1),
        # a prompt batch among many experts in groups, with the bias that balances them
        dict(name="route_16384x256_sigmoid_groups_top8", op="route", T=16384, E=256, k=8, dtype="fp32",
             score="sigmoid", bias=True, groups=8, top_groups=4),
        # one token decoded: the weights of its experts are the work
        dict(name="experts_1_of_64_top6_2048x1024", op="experts", T=1, E=64, k=6, D=2048, F=1024,
             dtype="bf16"),
        # a decode batch: most experts hold a token or two
        dict(name="experts_53_of_64_top8_4096x2048", op="experts", T=53, E=64, k=8, D=4096, F=2048,
             dtype="fp16"),
        # a prompt batch: hundreds of tokens an expert, unevenly
        dict(name="experts_4096_of_64_top8_4096x2048", op="experts", T=4096, E=64, k=8, D=4096, F=2048,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "route", "experts"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "quantize":
        rows, K = _log(rng, 1, 16384), 16 * _log(rng, 16, 512)
        return dict(op=op, rows=rows, K=K, dtype=rng.choice(["bf16", "fp16", "fp32"]) if rows <= 8192 else dtype,
                    layout=rng.choice(["permuted", "plain"]), encode=round(rng.uniform(0.5, 4.0), 2),
                    pad=rng.choice([0, 0, 8, 64]))
    if op == "gemm":
        return dict(op=op, N=_log(rng, 1, 4096), M=_log(rng, 200, 8192), K=32 * _log(rng, 8, 256),
                    L=rng.choice([1, 1, 2]), dtype=dtype, bias=rng.random() < 0.5,
                    act=rng.choice(["none", "silu", "gelu_tanh"]))
    if op == "route":
        if rng.random() < 0.5:
            return dict(op=op, T=_log(rng, 1, 16384), E=rng.randint(8, 256), k=rng.randint(1, 8),
                        dtype=rng.choice(["fp32", "bf16", "fp16"]), score="softmax", bias=False, groups=1,
                        top_groups=1)
        return dict(op=op, T=_log(rng, 1, 16384), E=8 * rng.randint(4, 32), k=rng.randint(1, 8), dtype="fp32",
                    score="sigmoid", bias=True, groups=8, top_groups=rng.randint(3, 8))
    return dict(op=op, T=_log(rng, 1, 2048), E=rng.choice([8, 24, 64]), k=rng.randint(1, 8),
                D=32 * _log(rng, 16, 128), F=32 * _log(rng, 8, 64), dtype=dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _codes(gen, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device=DEV, generator=gen)


def _scales(gen, rows, K, L):
    """Positive E4M3 codes of magnitudes 0.25 to 3.75, in 128x4 atoms with zero padding."""
    rm, rk = -(-rows // 128), -(-K // 64)
    s = torch.zeros((L, rm * 128, rk * 4), dtype=torch.uint8, device=DEV)
    s[:, :rows, : K // 16] = torch.randint(0x28, 0x48, (L, rows, K // 16), dtype=torch.uint8, device=DEV,
                                           generator=gen)
    return s.view(L, rm, 4, 32, rk, 4).permute(0, 1, 4, 3, 2, 5).contiguous().reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)
    s = dict(case)
    op = case["op"]
    if op == "quantize":
        # activations: unit rows of differing size with a few large channels
        x = torch.randn((case["rows"], case["K"] + case["pad"]), device=DEV, generator=gen)
        x *= torch.exp(0.5 * torch.randn((case["rows"], 1), device=DEV, generator=gen))
        x *= 1 + 20 * (torch.rand((1, case["K"] + case["pad"]), device=DEV, generator=gen) < 0.01)
        s["x"] = x.to(DTYPES[case["dtype"]])[:, : case["K"]]
    elif op == "gemm":
        N, M, K, L = (case[n] for n in "NMKL")
        s["a"], s["b"] = _codes(gen, L, M, K // 2), _codes(gen, L, N, K // 2)
        s["sfa"], s["sfb"] = _scales(gen, M, K, L), _scales(gen, N, K, L)
        s["alpha"] = 0.05 / math.sqrt(K)
        s["bias_t"] = torch.randn((L, M), device=DEV, generator=gen) if case["bias"] else None
    elif op == "route":
        T, E = case["T"], case["E"]
        s["logits"] = (2 * torch.randn((T, E), device=DEV, generator=gen)).to(DTYPES[case["dtype"]])
        s["bias_t"] = 0.05 * torch.randn((E,), device=DEV, generator=gen) if case["bias"] else None
    else:
        T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))
        s["x"] = torch.randn((T, D), device=DEV, generator=gen).to(DTYPES[case["dtype"]])
        # a learned router's uneven choices, its weights normalised
        score = torch.randn((T, E), device=DEV, generator=gen) + torch.randn((1, E), device=DEV, generator=gen)
        top = score.topk(k, dim=1)
        s["ids"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(top.values, dim=1)
        s["w1"], s["sf1"] = _codes(gen, E, 2 * F, D // 2), _scales(gen, 2 * F, D, E)
        s["w2"], s["sf2"] = _codes(gen, E, D, F // 2), _scales(gen, D, F, E)
        # per-expert weight scales over the activations' encode scales
        s["encode_x"], s["encode_h"] = 1.5, 2.0
        spread = torch.exp(0.1 * torch.randn((2, E), device=DEV, generator=gen))
        s["alpha1"] = spread[0] * (0.28 / math.sqrt(D) / s["encode_x"])
        s["alpha2"] = spread[1] * (0.28 / math.sqrt(F) / s["encode_h"])
    return s


# ---------------------------------------------------------------------------
# the plain form, fp32
# ---------------------------------------------------------------------------

def _plain_codes(q):
    """[..., K/2] bytes -> [..., K] fp32 values, the low nibble first."""
    v = torch.tensor(E2M1 + [-e for e in E2M1], device=q.device)
    pairs = torch.stack((v.repeat(16), v.repeat_interleave(16)), dim=1)
    return pairs[q.int()].flatten(-2)


def _plain_scales(sf, rows, K, L):
    """128x4 atoms -> [L, rows, K/16] fp32."""
    rm, rk = -(-rows // 128), -(-K // 64)
    s = sf.view(L, rm, rk, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(L, rm * 128, rk * 4)
    return s[:, :rows, : K // 16].contiguous().view(torch.float8_e4m3fn).float()


def _plain_matrix(q, s):
    return (_plain_codes(q).unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)


def _plain_quantize(y):
    """[..., K] fp32 -> values of the codes [..., K/16, 16], of the scales [..., K/16]."""
    y = y.unflatten(-1, (-1, 16))
    big = y.abs().amax(-1)
    # (a tensor as the divisor: a division by a number is a product with its rounded reciprocal on the GPU)
    s = (big / torch.full_like(big, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = y.abs() / torch.where(s > 0, s, torch.full_like(s, math.inf)).unsqueeze(-1)
    steps = ((r > 0.25).int() + (r >= 0.75).int() + (r > 1.25).int() + (r >= 1.75).int() + (r > 2.5).int()
             + (r >= 3.5).int() + (r > 5.0).int())
    return torch.tensor(E2M1, device=y.device)[steps] * torch.sign(y), s


def _plain_atoms(s, rows, K):
    """[rows, K/16] fp32 scale values -> E4M3 in 128x4 atoms, flat."""
    rm, rk = -(-rows // 128), -(-K // 64)
    full = torch.zeros((rm * 128, rk * 4), device=s.device)
    full[:rows, : K // 16] = s
    return full.view(rm, 4, 32, rk, 4).permute(0, 3, 2, 1, 4).reshape(-1).to(torch.float8_e4m3fn)


def _plain_activation(y, act):
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    if act == "gelu_tanh":
        return 0.5 * y * (1.0 + torch.tanh(0.7978845608028654 * (y + 0.044715 * y * y * y)))
    return y


def _plain_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["groups"]
    x = s["logits"].float()
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        score = e / e.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    rank = x if s["bias_t"] is None else score + s["bias_t"]
    if G > 1:
        best2 = (score if s["bias_t"] is None else rank).view(T, G, E // G).sort(2, descending=True).values[:, :, : min(2, E // G)].sum(2)
        keep = best2.sort(dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
        closed = torch.ones((T, G), dtype=torch.bool, device=x.device).scatter_(1, keep, False)
        rank = rank.masked_fill(closed.repeat_interleave(E // G, dim=1), -math.inf)
    ids = rank.sort(dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w}


def _plain_experts(s):
    T, k, D, F = s["T"], s["k"], s["D"], s["F"]
    xv, xs = _plain_quantize(s["x"].float() * s["encode_x"])
    x = (xv * xs.unsqueeze(-1)).flatten(-2)
    used, slot = torch.unique(s["ids"].long().flatten(), return_inverse=True)
    E = used.numel()
    # every expert's tokens in a row of the batch
    order = slot.argsort(stable=True)
    counts = torch.bincount(slot, minlength=E)
    at = torch.arange(T * k, device=DEV) - (counts.cumsum(0) - counts)[slot[order]]
    batch = torch.zeros((E, int(counts.max()), D), device=DEV)
    batch[slot[order], at] = x[order // k]
    w1 = _plain_matrix(s["w1"][used], _plain_scales(s["sf1"], 2 * F, D, s["E"])[used])
    u = torch.bmm(batch, w1.transpose(1, 2)) * s["alpha1"][used].view(-1, 1, 1)
    del w1, batch
    gate, up = u[:, :, 0::2], u[:, :, 1::2]
    hv, hs = _plain_quantize(gate / (1.0 + torch.exp(-gate)) * up * s["encode_h"])
    h = (hv * hs.unsqueeze(-1)).flatten(-2)
    w2 = _plain_matrix(s["w2"][used], _plain_scales(s["sf2"], D, F, s["E"])[used])
    y = torch.bmm(h, w2.transpose(1, 2)) * s["alpha2"][used].view(-1, 1, 1)
    rows = torch.empty((T * k, D), device=DEV)
    rows[order] = y[slot[order], at]
    out = (rows.view(T, k, D) * s["weights"].unsqueeze(-1)).sum(1)
    return {"out": out.to(s["x"].dtype)}


def _plain(s):
    op = s["op"]
    if op == "quantize":
        v, sc = _plain_quantize(s["x"].float() * s["encode"])
        x = ((v * sc.unsqueeze(-1)).flatten(-2) * (1.0 / s["encode"])).to(s["x"].dtype)
        scales = sc.to(torch.float8_e4m3fn) if s["layout"] == "plain" else _plain_atoms(sc, s["rows"], s["K"])
        return {"values": x, "scales": scales.flatten()}
    if op == "gemm":
        N, M, K, L = (s[n] for n in "NMKL")
        a = _plain_matrix(s["a"], _plain_scales(s["sfa"], M, K, L))
        b = _plain_matrix(s["b"], _plain_scales(s["sfb"], N, K, L))
        y = torch.bmm(b, a.transpose(1, 2)) * s["alpha"]
        if s["bias_t"] is not None:
            y = y + s["bias_t"].unsqueeze(1)
        return {"c": _plain_activation(y, s["act"]).to(DTYPES[s["dtype"]])}
    return _plain_route(s) if op == "route" else _plain_experts(s)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _calls(s):
    import nvfp4_block_scaled_gemv_gb300 as nv

    op = s["op"]
    if op == "quantize":
        layout = nv.SF_PLAIN if s["layout"] == "plain" else nv.SF_PERMUTED_128x4
        q, sf = nv.quantize(s["x"], encode_scale=s["encode"], sf_layout=layout)
        x = nv.dequantize(q, sf, scale=1.0 / s["encode"], dtype=s["x"].dtype, sf_layout=layout)
        return {"values": x, "scales": sf.flatten().view(torch.float8_e4m3fn)}
    if op == "gemm":
        act = {"none": nv.ACT_NONE, "silu": nv.ACT_SILU, "gelu_tanh": nv.ACT_GELU_TANH}[s["act"]]
        return {"c": nv.gemm(s["a"], s["b"], s["sfa"], s["sfb"], alpha=s["alpha"], bias=s["bias_t"],
                             activation=act, dtype=DTYPES[s["dtype"]])}
    if op == "route":
        score = nv.SCORE_SOFTMAX if s["score"] == "softmax" else nv.SCORE_SIGMOID
        ids, weights = nv.route(s["logits"], s["k"], score=score, bias=s["bias_t"], groups=s["groups"],
                                top_groups=s["top_groups"], renormalize=True)
        return {"ids": ids, "weights": weights}
    return {"out": nv.moe_ffn(s["x"], s["ids"], s["weights"], s["w1"], s["sf1"], s["w2"], s["sf2"],
                              alpha1=s["alpha1"], alpha2=s["alpha2"], encode_x=s["encode_x"],
                              encode_h=s["encode_h"])}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e exactly, by a table (a power function on the GPU rounds)."""
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=e.device)[e.long() + 160]


def _decode64(q):
    c = torch.stack((q % 16, q // 16), dim=-1).flatten(-2).to(torch.int16)
    e, m, sign = c // 2 % 4, c % 2, 1.0 - 2.0 * (c // 8).double()
    return sign * torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * _two_to(e - 1))


def _scale64(b):
    b = b.to(torch.int16)
    e, m = b // 8 % 16, (b % 8).double()
    return torch.where(e == 0, m / 512, (1 + m / 8) * _two_to(e - 7))


def _matrix64(q, sf, rows, K, L):
    """One batch's dense matrix at a time, the scale bytes found by their address."""
    rm, rk = -(-rows // 128), -(-K // 64)
    m, kb = torch.arange(rows, device=q.device).view(-1, 1), torch.arange(K // 16, device=q.device)
    at = ((m // 128) * rk + kb // 4) * 512 + m % 32 * 16 + m // 32 % 4 * 4 + kb % 4
    for i in range(L):
        sc = _scale64(sf[i * rm * rk * 512:(i + 1) * rm * rk * 512][at])
        yield _decode64(q[i]) * sc.repeat_interleave(16, dim=1)


def _quantize64(y):
    y = y.unflatten(-1, (-1, 16))
    big = y.abs().amax(-1)
    big = (big / torch.full_like(big, 6.0)).clamp(max=448)
    step = _two_to(torch.frexp(big).exponent.clamp(min=-5) - 4)
    s = torch.round(big / step) * step
    r = (y / torch.where(s > 0, s, torch.full_like(s, math.inf)).unsqueeze(-1)).clamp(-6, 6)
    fine = torch.where(r.abs() < 2, 0.5, torch.where(r.abs() < 4, 1.0, 2.0))
    return torch.round(r / fine) * fine, s


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        v, sc = _quantize64(s["x"].double() * case["encode"])
        x = (v * sc.unsqueeze(-1)).flatten(-2) / case["encode"]
        if case["layout"] == "permuted":
            rm, rk = -(-rows // 128), -(-K // 64)
            m, kb = torch.arange(rows, device=DEV).view(-1, 1), torch.arange(K // 16, device=DEV)
            flat = torch.zeros(rm * rk * 512, dtype=torch.float64, device=DEV)
            flat[((m // 128) * rk + kb // 4) * 512 + m % 32 * 16 + m // 32 % 4 * 4 + kb % 4] = sc
            sc = flat
        return {"values": x, "scales": sc.flatten()}
    if op == "gemm":
        N, M, K, L = (case[n] for n in "NMKL")
        c = torch.empty((L, N, M), dtype=torch.float64, device=DEV)
        for i, (a, b) in enumerate(zip(_matrix64(s["a"], s["sfa"], M, K, L), _matrix64(s["b"], s["sfb"], N, K, L))):
            y = b @ a.T * s["alpha"] + (0 if s["bias_t"] is None else s["bias_t"][i].double())
            if case["act"] == "silu":
                y = y * torch.sigmoid(y)
            elif case["act"] == "gelu_tanh":
                y = y * torch.sigmoid(math.sqrt(8 / math.pi) * (y + 0.044715 * y ** 3))
            c[i] = y
        return {"c": c}
    if op == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
        x = s["logits"].double()
        score = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
        rank = x if s["bias_t"] is None else score + s["bias_t"].double()
        if G > 1:
            best = (score if s["bias_t"] is None else rank).view(T, G, E // G).topk(min(2, E // G), dim=2).values.sum(2)
            kept = best.argsort(dim=1, descending=True, stable=True)[:, : case["top_groups"]]
            mine = (torch.arange(E, device=DEV) // (E // G)).view(1, E, 1)
            rank = torch.where((mine == kept.unsqueeze(1)).any(2), rank, -math.inf)
        w = score.gather(1, rank.argsort(dim=1, descending=True, stable=True)[:, :k])
        return {"ids": None, "weights": w / w.sum(1, keepdim=True)}
    T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))
    v, sc = _quantize64(s["x"].double() * s["encode_x"])
    x = (v * sc.unsqueeze(-1)).flatten(-2)
    out = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    both = zip(_matrix64(s["w1"], s["sf1"], 2 * F, D, E), _matrix64(s["w2"], s["sf2"], D, F, E))
    for e, (w1, w2) in enumerate(both):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        u = x[t] @ w1.T * s["alpha1"][e].double()
        v, sc = _quantize64(u[:, 0::2] * torch.sigmoid(u[:, 0::2]) * u[:, 1::2] * s["encode_h"])
        y = (v * sc.unsqueeze(-1)).flatten(-2) @ w2.T * s["alpha2"][e].double()
        out.index_add_(0, t, y * s["weights"][t, j].double().unsqueeze(1))
    return {"out": out}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def _matrix_bytes(rows, K):
    return rows * (K // 2 + K // 16)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        # both calls: the rows read, codes and scales written, read again, the rows written
        return {"bytes": 2 * rows * K * size + 2 * _matrix_bytes(rows, K), "flops": 4 * rows * K}
    if op == "gemm":
        N, M, K, L = (case[n] for n in "NMKL")
        return {"bytes": L * (_matrix_bytes(M, K) + _matrix_bytes(N, K) + N * M * size + (4 * M if case["bias"] else 0)),
                "flops": 2 * L * N * M * K}
    if op == "route":
        return {"bytes": case["T"] * (case["E"] * size + 8 * case["k"]) + (4 * case["E"] if case["bias"] else 0),
                "flops": 8 * case["T"] * case["E"]}
    T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))
    # experts that get a token when the choices are even: E (1 - (1 - k/E)^T)
    used = E * (1 - (1 - k / E) ** T) if k < E else E
    return {"bytes": used * (_matrix_bytes(2 * F, D) + _matrix_bytes(D, F)) + 2 * T * D * size + 8 * T * k,
            "flops": 2 * T * k * 3 * F * D}
