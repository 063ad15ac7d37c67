"""The operators of attention on a 4-bit cache, as a program that serves a model calls them.

Three operators that follow each other in a layer, each with its plain form:

  rope       rotary positions of query and key heads
  cache      keys and values quantised into pages of a cache, and read back
  attention  queries against the keys and values of such a cache

``own`` chooses between the plain form (elementary torch operations in fp32,
angles in fp64) and the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def listed():
    return [
        # one token decoded: its query and key heads, in the fused projection's row
        dict(name="rope_1x40x128_bf16", op="rope", T=1, H=40, D=128, rot=128, interleaved=False, scaling="none",
             far=8000, inverse=False, pad=1024, dtype="bf16"),
        # part of the head, interleaved pairs, positions far beyond the trained context
        dict(name="rope_333x27x128_part_interleaved_fp16", op="rope", T=333, H=27, D=128, rot=96, interleaved=True,
             scaling="ramp", far=1000000, inverse=False, pad=8, dtype="fp16"),
        # a full batch of prompts
        dict(name="rope_16384x40x128_bf16", op="rope", T=16384, H=40, D=128, rot=128, interleaved=False,
             scaling="bands", far=131072, inverse=False, pad=1024, dtype="bf16"),
        # the gradient of the rotation, 32-bit
        dict(name="rope_2047x16x64_inverse_fp32", op="rope", T=2047, H=16, D=64, rot=64, interleaved=False,
             scaling="linear", far=4096, inverse=True, pad=0, dtype="fp32"),
        # a decode batch: a row of each sequence
        dict(name="cache_24x8x128_bf16", op="cache", T=24, H=8, D=128, page=64, encode=False, pad=0, skip=0,
             dtype="bf16"),
        # a ragged prompt in small pages, scaled heads, strided rows, some of them padding
        dict(name="cache_777x5x64_fp16", op="cache", T=777, H=5, D=64, page=16, encode=True, pad=40, skip=9,
             dtype="fp16"),
        # a full batch of prompts
        dict(name="cache_16384x8x128_bf16", op="cache", T=16384, H=8, D=128, page=64, encode=True, pad=0, skip=0,
             dtype="bf16"),
        # one token of one short sequence: launch latency
        dict(name="attention_1x1_len900_bf16", op="attention", B=1, n=1, ragged=False, lo=900, hi=900, Hq=32, Hkv=8,
             D=128, page=64, window=0, dtype="bf16"),
        # a decode batch of very different lengths, an odd group of heads, small pages, a window
        dict(name="attention_45x1_len17to9000_window_fp16", op="attention", B=45, n=1, ragged=False, lo=17, hi=9000,
             Hq=30, Hkv=6, D=64, page=16, window=4096, dtype="fp16"),
        # drafted tokens verified together, wide heads
        dict(name="attention_8x4_len500to12000_bf16", op="attention", B=8, n=4, ragged=False, lo=500, hi=12000,
             Hq=16, Hkv=4, D=256, page=32, window=0, dtype="bf16"),
        # a decode batch of long contexts: the cache's bytes are the work
        dict(name="attention_32x1_len16kto32k_bf16", op="attention", B=32, n=1, ragged=False, lo=16384, hi=32768,
             Hq=64, Hkv=8, D=128, page=64, window=0, dtype="bf16"),
        # prompts of different lengths after cached prefixes
        dict(name="attention_4x4096_ragged_len4kto16k_bf16", op="attention", B=4, n=4096, ragged=True, lo=4200,
             hi=16000, Hq=32, Hkv=8, D=128, page=64, window=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "cache", "attention", "attention"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        D = rng.choice([64, 96, 128, 256])
        return dict(op=op, T=_log(rng, 1, 8192), H=rng.randint(1, 40), D=D,
                    rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "base", "ramp", "bands"]), far=_log(rng, 100, 1000000),
                    inverse=rng.random() < 0.3, pad=rng.choice([0, 8, 1024]),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]))
    if op == "cache":
        return dict(op=op, T=_log(rng, 1, 8192), H=rng.randint(1, 16), D=rng.choice([64, 128, 256]),
                    page=rng.choice([16, 32, 64, 128]), encode=rng.random() < 0.5, pad=rng.choice([0, 8, 40]),
                    skip=rng.choice([0, 0, 5]), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    Hkv, group, D = rng.randint(1, 8), rng.randint(1, 8), rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if rng.random() < 0.6:
        n, B, hi = rng.choice([1, 1, 1, 2, 4, 7]), _log(rng, 1, 64), _log(rng, 64, 16384)
        return dict(op=op, B=B, n=n, ragged=False, lo=max(n, hi // rng.choice([1, 3, 20])), hi=hi, Hq=group * Hkv,
                    Hkv=Hkv, D=D, page=page, window=rng.choice([0, 0, 512]), dtype=dtype)
    n, B = _log(rng, 16, 2048), rng.randint(1, 4)
    hi = n + _log(rng, 1, 8192)
    return dict(op=op, B=B, n=n, ragged=rng.random() < 0.7, lo=n, hi=hi, Hq=group * Hkv, Hkv=Hkv, D=D, page=page,
                window=rng.choice([0, 0, 512]), dtype=dtype)


def _spread(lo, hi, count):
    """count whole numbers from lo to hi."""
    return [hi] if count == 1 else [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _shape(case):
    """A batch's lengths and query counts, the longest first."""
    lens = _spread(case["lo"], case["hi"], case["B"])[::-1]
    n = _spread(max(1, case["n"] // 8), case["n"], case["B"])[::-1] if case["ragged"] else [case["n"]] * case["B"]
    return lens, n


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _rows(gen, T, H, D):
    """Heads of unit size, a few channels of each far larger."""
    x = torch.randn((T, H, D), device=DEV, generator=gen)
    return x * (1 + 4 * (torch.rand((1, H, D), device=DEV, generator=gen) < 0.02))


def _pack(k, v, page):
    """Quantised k and v [tokens, H, D] -> pages [P, H, page/16, 2, D/64, 16 * 36]: per 16 tokens and
    64 elements, the tokens' 32 bytes of codes and then their 4 scale bytes each."""
    out = []
    for x in (k, v):
        T, H, D = x.shape
        y = x.float().unflatten(-1, (-1, 16))
        s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
        r = y.abs() / torch.where(s.float() > 0, s.float(), torch.full_like(s.float(), math.inf)).unsqueeze(-1)
        c = torch.bucketize(r, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)).to(torch.uint8)
        c = (c + 8 * (y < 0).to(torch.uint8)).flatten(-2)
        q = c[..., 0::2] + 16 * c[..., 1::2]
        q = q.view(T // page, page // 16, 16, H, D // 64, 32).permute(0, 3, 1, 4, 2, 5)
        s = s.view(torch.uint8).view(T // page, page // 16, 16, H, D // 64, 4).permute(0, 3, 1, 4, 2, 5)
        out.append(torch.cat((q.flatten(-2), s.flatten(-2)), dim=-1))
    return torch.stack(out, dim=3)


def _scaling(case):
    return {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
            "ramp": dict(factor=32.0, original=4096, low=1.0, high=32.0),
            "bands": dict(factor=8.0, original=8192, low=1.0, high=4.0)}[case["scaling"]]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)
    rng = random.Random(int(seed) * 7919 + 31)
    s = dict(case)
    dtype, op = DTYPES[case["dtype"]], case["op"]
    if op == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        x = torch.randn((T, H * D + case["pad"]), device=DEV, generator=gen).to(dtype)
        s["x"] = x[:, : H * D].unflatten(1, (H, D))
        s["positions"] = torch.randint(0, case["far"], (T,), dtype=torch.int32, device=DEV, generator=gen)
        s["factor"] = 1.0 + 0.1 * math.log(32.0) if case["scaling"] == "ramp" else 1.0
        if own:
            import nvfp4_block_scaled_gemv_gb300 as nv

            s["table"] = nv.rope_table(case["rot"], base=10000.0, scaling=case["scaling"], device=DEV, **_scaling(case))
    elif op == "cache":
        T, H, D, page = case["T"], case["H"], case["D"], case["page"]
        kv = torch.randn((2, T, H * D + case["pad"]), device=DEV, generator=gen)
        kv *= torch.exp(0.5 * torch.randn((2, T, 1), device=DEV, generator=gen))
        s["k"], s["v"] = kv.to(dtype)[:, :, : H * D].unflatten(2, (H, D)).unbind(0)
        pages = -(-T // page) + 3
        slots = torch.randperm(pages * page, device=DEV, generator=gen)[:T]
        if case["skip"]:
            slots[:: case["skip"]] = -1
        s["slots"], s["pages"] = slots, pages
        scale = torch.exp(0.5 * torch.randn((2, H), device=DEV, generator=gen))
        s["encode_k"], s["encode_v"] = (scale[0].contiguous(), scale[1].contiguous()) if case["encode"] else (None, None)
        if own:
            s["cache"] = torch.zeros((pages, H, page // 16, 2, D // 64, 576), dtype=torch.uint8, device=DEV)
        else:
            s["cache"] = torch.zeros((2, pages * page, H, D), device=DEV)
    else:
        B, Hq, Hkv, D, page = (case[n] for n in ("B", "Hq", "Hkv", "D", "page"))
        lens, counts = _shape(case)
        order = list(range(B))
        rng.shuffle(order)
        s["lens"], s["counts"] = [lens[i] for i in order], [counts[i] for i in order]
        used = [-(-n // page) for n in s["lens"]]
        total = sum(used) + 2
        s["cache"] = torch.empty((total, Hkv, page // 16, 2, D // 64, 576), dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 26) // (page * Hkv * D))
        for p in range(0, total, step):
            t = min(step, total - p) * page
            s["cache"][p: p + step] = _pack(_rows(gen, t, Hkv, D), _rows(gen, t, Hkv, D), page)
        at = torch.randperm(total, device=DEV, generator=gen).to(torch.int32)
        s["table"] = torch.zeros((B, max(used)), dtype=torch.int32, device=DEV)
        for b, n in enumerate(used):
            s["table"][b, :n] = at[sum(used[:b]): sum(used[:b]) + n]
        T = sum(s["counts"])
        s["q"] = torch.randn((T, Hq, D), device=DEV, generator=gen).to(dtype)
        s["lengths"] = torch.tensor(s["lens"], dtype=torch.int32, device=DEV)
        starts = [0]
        for n in s["counts"]:
            starts.append(starts[-1] + n)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV) if case["ragged"] else None
        spread = torch.exp(0.2 * torch.randn((2, Hkv), device=DEV, generator=gen))
        s["encode_k"], s["encode_v"] = spread[0].contiguous(), spread[1].contiguous()
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

def _frequencies(case):
    """Radians per position of each pair."""
    rot, base, kind, o = case["rot"], 10000.0, case["scaling"], _scaling(case)
    if kind == "base":
        base *= o["factor"] ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if kind == "linear":
            f /= o["factor"]
        elif kind == "ramp":
            # pairs that turn often within the original length stay, those that turn rarely are stretched
            first, last = (rot * math.log(o["original"] / (turns * 2 * math.pi)) / (2 * math.log(base))
                           for turns in (o["high"], o["low"]))
            first, last = max(math.floor(first), 0), min(math.ceil(last), rot - 1)
            part = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            f = f / o["factor"] * part + f * (1 - part)
        elif kind == "bands":
            turns = o["original"] * f / (2 * math.pi)
            part = min(max((turns - o["low"]) / (o["high"] - o["low"]), 0.0), 1.0)
            f = f * part + f / o["factor"] * (1 - part)
        out.append(f)
    return out


def _plain_rope(s):
    rot = s["rot"]
    angle = s["positions"].double().unsqueeze(1) * torch.tensor(_frequencies(s), dtype=torch.float64, device=DEV)
    cos, sin = (f(angle).float().unsqueeze(1) * s["factor"] for f in (torch.cos, torch.sin))
    if s["inverse"]:
        sin = -sin
    x = s["x"].float()
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), dim=-1)
    return {"y": torch.cat((y, x[..., rot:]), dim=-1).to(s["x"].dtype)}


def _plain_quantized(x, encode):
    """The values that x [T, H, D] fp32 keeps in 4 bits."""
    if encode is not None:
        x = x * encode.view(1, -1, 1)
    y = x.unflatten(-1, (-1, 16))
    big = y.abs().amax(-1)
    # (a tensor as the divisor: a division by a number is a product with its rounded reciprocal on the GPU)
    sc = (big / torch.full_like(big, 6.0)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    r = y.abs() / torch.where(sc > 0, sc, torch.full_like(sc, math.inf)).unsqueeze(-1)
    steps = ((r > 0.25).int() + (r >= 0.75).int() + (r > 1.25).int() + (r >= 1.75).int() + (r > 2.5).int()
             + (r >= 3.5).int() + (r > 5.0).int())
    return (torch.tensor(E2M1, device=DEV)[steps] * torch.sign(y) * sc.unsqueeze(-1)).flatten(-2)


def _plain_cache(s):
    slots, out = s["slots"], {}
    mine = slots >= 0
    for i, n in enumerate("kv"):
        values = _plain_quantized(s[n].float(), s["encode_" + n])
        s["cache"][i, slots[mine]] = values[mine]
        got = s["cache"][i, slots.clamp(min=0)] * mine.view(-1, 1, 1)
        if s["encode_" + n] is not None:
            got = got * (1.0 / s["encode_" + n]).view(1, -1, 1)
        out[n] = got.to(s[n].dtype)
    return out


def _plain_tokens(s, b):
    """k, v [len, Hkv, D] fp32 of a sequence."""
    n, D, page = s["lens"][b], s["D"], s["page"]
    c = s["cache"][s["table"][b, : -(-n // page)].long()]
    codes = c[..., :512].unflatten(-1, (16, 32))
    value = torch.tensor(E2M1 + [-e for e in E2M1], device=DEV)
    x = torch.stack((value[(codes & 15).int()], value[(codes >> 4).int()]), dim=-1).flatten(-2).unflatten(-1, (4, 16))
    x = x * c[..., 512:].unflatten(-1, (16, 4)).contiguous().view(torch.float8_e4m3fn).float().unsqueeze(-1)
    # [pages, H, granules, 2, planes, tokens, 4, 16]
    x = x.permute(3, 0, 2, 5, 1, 4, 6, 7).reshape(2, -1, s["Hkv"], D)[:, :n]
    return x[0] * (1.0 / s["encode_k"]).view(1, -1, 1), x[1] * (1.0 / s["encode_v"]).view(1, -1, 1)


def _plain_attention(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    out = torch.empty((s["q"].shape[0], Hq, D), dtype=s["q"].dtype, device=DEV)
    lse = torch.empty((s["q"].shape[0], Hq), device=DEV)
    at = 0
    for b, (length, n) in enumerate(zip(s["lens"], s["counts"])):
        k, v = _plain_tokens(s, b)
        q = s["q"][at: at + n].float().unflatten(1, (Hkv, Hq // Hkv)).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
        score = torch.bmm(q, k.permute(1, 2, 0)) * (1.0 / math.sqrt(D))
        here = torch.arange(length - n, length, device=DEV).view(1, -1, 1)
        there = torch.arange(length, device=DEV)
        seen = there <= here
        if s["window"]:
            seen = seen & (there > here - s["window"])
        score = score.unflatten(1, (-1, n)).masked_fill(~seen, -math.inf).flatten(1, 2)
        top = score.amax(2, keepdim=True)
        p = torch.exp(score - top)
        total = p.sum(2, keepdim=True)
        y = torch.bmm(p, v.transpose(0, 1)) / total
        out[at: at + n] = y.view(Hkv, -1, n, D).permute(2, 0, 1, 3).reshape(n, Hq, D).to(out.dtype)
        lse[at: at + n] = (top + torch.log(total)).view(Hkv, -1, n).permute(2, 0, 1).reshape(n, Hq)
        at += n
    return {"out": out, "lse": lse}


def _plain(s):
    return {"rope": _plain_rope, "cache": _plain_cache, "attention": _plain_attention}[s["op"]](s)


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _calls(s):
    import nvfp4_block_scaled_gemv_gb300 as nv

    if s["op"] == "rope":
        return {"y": nv.rope(s["x"], s["positions"], s["table"], interleaved=s["interleaved"], factor=s["factor"],
                             inverse=s["inverse"])}
    if s["op"] == "cache":
        nv.kv_write(s["k"], s["v"], s["cache"], s["slots"], encode_k=s["encode_k"], encode_v=s["encode_v"])
        k, v = nv.kv_read(s["cache"], s["slots"], dtype=s["k"].dtype, encode_k=s["encode_k"], encode_v=s["encode_v"])
        return {"k": k, "v": v}
    out, lse = nv.attention(s["q"], s["cache"], s["table"], s["lengths"], q_starts=s["starts"], max_q=s["n"],
                            window=s["window"], encode_k=s["encode_k"], encode_v=s["encode_v"], return_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    return _calls(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _two_to(e):
    """2^e exactly, by a table (a power function on the GPU rounds)."""
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device=e.device)[e.long() + 160]


def _exact_rope(s):
    rot, freq = s["rot"], torch.tensor(_frequencies(s), dtype=torch.float64, device=DEV)
    angle = s["positions"].double().view(-1, 1, 1) * freq
    turn = torch.polar(torch.full_like(angle, s["factor"]), -angle if s["inverse"] else angle)
    x = s["x"].double()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if s["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return {"y": y}


def _exact_cache(s):
    out = {}
    for n in "kv":
        encode = torch.ones(s["H"], device=DEV) if s["encode_" + n] is None else s["encode_" + n]
        # (the scaled value is an fp32 number, by definition)
        y = (s[n].float() * encode.view(1, -1, 1)).double().unflatten(-1, (-1, 16))
        big = y.abs().amax(-1)
        big = (big / torch.full_like(big, 6.0)).clamp(max=448)
        step = _two_to(torch.frexp(big).exponent.clamp(min=-5) - 4)
        sc = (torch.round(big / step) * step).unsqueeze(-1)
        r = (y / torch.where(sc > 0, sc, torch.full_like(sc, math.inf))).clamp(-6, 6)
        fine = torch.where(r.abs() < 2, 0.5, torch.where(r.abs() < 4, 1.0, 2.0))
        x = (torch.round(r / fine) * fine * sc).flatten(-2) / encode.double().view(1, -1, 1)
        out[n] = torch.where((s["slots"] < 0).view(-1, 1, 1), 0.0, x)
    return out


def _exact_side(s, b, side, h):
    """[len, D] of one head of a sequence, every byte found by its address."""
    n, D, page = s["lens"][b], s["D"], s["page"]
    t, d = torch.arange(n, device=DEV).view(-1, 1), torch.arange(D, device=DEV)
    planes, flat = D // 64, s["cache"].view(-1)
    granule = (s["table"][b].long()[t // page] * s["Hkv"] + h) * (page // 16) + t % page // 16
    plane = ((granule * 2 + side) * planes + d // 64) * 576
    byte = flat[plane + t % 16 * 32 + d % 64 // 2].to(torch.int16)
    c = torch.where(d % 2 == 1, byte // 16, byte % 16)
    e, m = c // 2 % 4, c % 2
    code = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * _two_to(e - 1)) * (1.0 - 2.0 * (c // 8).double())
    byte = flat[plane + 512 + t % 16 * 4 + d % 64 // 16].to(torch.int16)
    e, m = byte // 8 % 16, (byte % 8).double()
    return code * torch.where(e == 0, m / 512, (1 + m / 8) * _two_to(e - 7))


def _exact_attention(s):
    Hq, Hkv, D = s["Hq"], s["Hkv"], s["D"]
    G = Hq // Hkv
    out = torch.empty((s["q"].shape[0], Hq, D), dtype=torch.float64, device=DEV)
    lse = torch.empty((s["q"].shape[0], Hq), dtype=torch.float64, device=DEV)
    at = 0
    for b, (length, n) in enumerate(zip(s["lens"], s["counts"])):
        far = torch.arange(n, device=DEV).view(-1, 1, 1) + length - n - torch.arange(length, device=DEV)
        seen = (far >= 0) & (far < (s["window"] or length + 1))
        for h in range(Hkv):
            k, v = (_exact_side(s, b, i, h) / s[e][h].double() for i, e in ((0, "encode_k"), (1, "encode_v")))
            rows = slice(h * G, h * G + G)
            score = s["q"][at: at + n, rows].double() @ k.T / math.sqrt(D)
            score = torch.where(seen, score, -math.inf)
            lse[at: at + n, rows] = torch.logsumexp(score, 2)
            out[at: at + n, rows] = torch.softmax(score, 2) @ v
        at += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "attention": _exact_attention}[case["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case["dtype"]]
    if op == "rope":
        return {"bytes": case["T"] * (case["H"] * case["D"] * 2 * size + 4), "flops": case["T"] * case["H"] * case["rot"] * 3}
    if op == "cache":
        # both calls: rows read, codes and scales written, read again, rows written
        values = 2 * case["T"] * case["H"] * case["D"]
        return {"bytes": values * 2 * size + values * 9 // 8 + 16 * case["T"], "flops": 4 * values}
    Hq, Hkv, D, window = case["Hq"], case["Hkv"], case["D"], case["window"]
    tokens = pairs = queries = 0
    for length, n in zip(*_shape(case)):
        first = max(0, length - n - window + 1) if window else 0
        tokens += length - first
        queries += n
        if window:
            pairs += sum(min(p + 1, window) for p in range(length - n, length))
        else:
            pairs += n * (length - n) + n * (n + 1) // 2
    return {"bytes": tokens * Hkv * D * 9 // 8 + queries * Hq * (2 * D * size + 4), "flops": 4 * pairs * Hq * D}
