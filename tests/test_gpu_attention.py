"""The attention operators on a GPU against their definitions in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402
from oracle import attention as oa  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {n: torch.finfo(t).eps / 2 for n, t in DT.items()}
TINY = {"fp16": 2.0 ** -25, "bf16": 0.0, "fp32": 0.0}  # half a step of the smallest numbers


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def host(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

def rope_bound(x, want, table, interleaved, factor, dtype):
    """The result's rounding, and in fp32: cosine and sine within 2^-22 (the angle's 2^-25 of an eighth
    turn, sincospi's 2 ulp, the factor's product), two products and a sum."""
    n = len(table)
    i = np.arange(n)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, n + i)
    size = np.zeros_like(want)
    size[..., first] = size[..., second] = np.abs(x[..., first]) + np.abs(x[..., second])
    return HALF[dtype] * np.abs(want) * (1 + 2.0 ** -10) + TINY[dtype] + 2.0 ** -21 * abs(factor) * size


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,D,rot,pad", [(1, 1, 2, 2, 0), (1, 40, 128, 128, 0), (7, 3, 64, 64, 8), (33, 5, 96, 24, 1),
                                           (130, 2, 80, 30, 0), (5, 9, 256, 128, 16), (3, 2, 1030, 1024, 0),
                                           (600, 1, 17, 4, 0), (2000, 4, 64, 48, 0)])
def test_rope(T, H, D, rot, pad, dtype, interleaved, inverse):
    rng = np.random.default_rng(T + D)
    x = torch.from_numpy(rng.standard_normal((T, H * D + pad)).astype(np.float32)).to(DT[dtype])
    pos = np.concatenate(([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1000003, 131071],
                          rng.integers(-5000, 1 << 20, T)))[:T].astype(np.int32)
    rng.shuffle(pos)
    table = nv.rope_table(rot, base=500000.0)
    xd = x.to(DEV)[:, : H * D].unflatten(1, (H, D))
    y = nv.rope(xd, gpu(pos), table, interleaved=interleaved, factor=1.25, inverse=inverse)
    xv = host(xd)
    want = oa.rope(xv, pos, table.tolist(), interleaved, 1.25, inverse)
    assert y.shape == (T, H, D) and y.is_contiguous()
    assert (np.abs(host(y) - want) <= rope_bound(xv, want, table, interleaved, 1.25, dtype)).all()
    assert torch.equal(y[..., rot:], xd[..., rot:])
    # in place, in the wider buffer, whose other elements stay
    buffer = x.to(DEV)
    view = buffer[:, : H * D].unflatten(1, (H, D))
    assert nv.rope(view, gpu(pos), table, interleaved=interleaved, factor=1.25, inverse=inverse, out=view) is view
    assert torch.equal(view, y) and torch.equal(buffer[:, H * D:], x.to(DEV)[:, H * D:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient_is_the_inverse_rotation(interleaved):
    """<rope(x), g> has the gradient rope(g, inverse): the formula's, and that of differences."""
    rng = np.random.default_rng(3)
    T, H, D, rot = 9, 2, 32, 20
    x, g = rng.standard_normal((2, T, H, D)).astype(np.float32)
    pos = rng.integers(0, 1 << 20, T).astype(np.int32)
    table = nv.rope_table(rot)
    grad = host(nv.rope(gpu(g), gpu(pos), table, interleaved=interleaved, factor=1.5, inverse=True))

    def loss(x):
        return (oa.rope(x, pos, table.tolist(), interleaved, 1.5) * g).sum()

    for _ in range(40):
        at = tuple(rng.integers(0, n) for n in x.shape)
        step = np.zeros(x.shape)
        step[at] = 2.0 ** -10
        diff = (loss(x + step) - loss(x - step)) / 2.0 ** -9  # (linear: exact but for fp64's rounding)
        # two products with cosines within 2^-22 of |g| <= 5, and a sum
        assert abs(diff - grad[at]) <= 2.0 ** -21 * 1.5 * 10
    back = nv.rope(nv.rope(gpu(x), gpu(pos), table, interleaved=interleaved, factor=2.0), gpu(pos), table,
                   interleaved=interleaved, factor=0.5, inverse=True)
    assert np.abs(host(back)[..., :rot] - x[..., :rot]).max() <= 2.0 ** -19 * np.abs(x).max()


def test_rope_turns_only_the_heads_given():
    """Query and key heads of a fused row in one call, into another buffer of the same rows."""
    rng = np.random.default_rng(4)
    row = gpu(rng.standard_normal((12, 10 * 64)).astype(np.float32)).bfloat16()
    pos, table = gpu(np.arange(12, dtype=np.int32)), nv.rope_table(64)
    heads = row.unflatten(1, (10, 64))
    want = nv.rope(heads[:, 2:5].contiguous(), pos, table)
    before = row.clone()
    got = nv.rope(heads[:, 2:5], pos, table, out=heads[:, 6:9])
    assert torch.equal(got, want) and torch.equal(heads[:, :6], before.unflatten(1, (10, 64))[:, :6])
    assert torch.equal(heads[:, 9:], before.unflatten(1, (10, 64))[:, 9:])
    with pytest.raises(ValueError):
        nv.rope(heads[:, 2:5], pos, table, out=heads[:, 4:7])
    assert nv.rope(heads[:0], pos[:0], table).shape == (0, 10, 64)


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("T,H,D,page,pad,encode", [(1, 1, 64, 16, 0, False), (9, 3, 128, 32, 0, True),
                                                   (70, 2, 256, 16, 3, True), (333, 5, 64, 48, 40, False),
                                                   (40, 8, 128, 64, 8, True)])
def test_cache_write_and_read(T, H, D, page, pad, encode, dtype):
    rng = np.random.default_rng(T + D)
    x = rng.standard_normal((2, T, H * D + pad)) * np.exp(3 * rng.standard_normal((2, T, 1)))
    x[:, :, ::37] *= 50
    x[0, :, :16] = 0
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[::7] = rng.choice([-1, -(1 << 62), pages * page, 1 << 40], slots[::7].shape)
    e = np.exp2(rng.integers(-3, 4, (2, H))).astype(np.float32) * np.float32(1.37) if encode else (None, None)
    ed = [None if v is None else gpu(v) for v in e]
    kd, vd = t.to(DEV)[:, :, : H * D].unflatten(2, (H, D)).unbind(0)
    cache = torch.full((pages, H, page // 16, 2, D // 64, 576), 0x5A, dtype=torch.uint8, device=DEV)
    assert nv.kv_write(kd, vd, cache, gpu(slots), encode_k=ed[0], encode_v=ed[1]) is cache
    want = oa.empty_cache(pages, H, D, page, fill=0x5A)
    kv = [v.float().cpu().numpy() for v in (kd, vd)]
    oa.write(want, slots, *kv, *e)
    got = cache.cpu().numpy()
    assert np.array_equal(got, want)  # (codes, scales, and every byte of other slots)
    # back, in every type: one product with the reciprocal in fp32, one rounding
    vals = oa.values(want)
    there = (slots >= 0) & (slots < pages * page)
    for out in DT:
        back = nv.kv_read(cache, gpu(slots), dtype=DT[out], encode_k=ed[0], encode_v=ed[1])
        for side in range(2):
            r = np.float32(1.0) if e[side] is None else (np.float32(1.0) / e[side])[:, None]
            f = np.where(there[:, None, None], vals[side][np.where(there, slots, 0)], 0).astype(np.float32) * r
            # (an fp16 input may hold infinities: their blocks are NaN on both sides)
            torch.testing.assert_close(back[side].cpu(), torch.from_numpy(f.astype(np.float32)).to(DT[out]), rtol=0,
                                       atol=0, equal_nan=True)


def test_cache_keeps_nan_and_infinity_in_their_blocks():
    x = torch.ones(3, 1, 64)
    x[0, 0, 20], x[1, 0, 40], x[2, 0, 0] = float("inf"), float("nan"), 1e-20
    cache = nv.kv_cache(1, 1, 64, 16, device=DEV)
    slots = torch.arange(3, device=DEV)
    nv.kv_write(x.to(DEV), x.to(DEV), cache, slots)
    k, v = nv.kv_read(cache, slots)
    assert torch.equal(k.isnan(), v.isnan())
    bad = torch.zeros(3, 64, dtype=torch.bool)
    bad[0, 16:32] = bad[1, 32:48] = True
    assert torch.equal(k[:, 0].isnan().cpu(), bad)
    assert (k[:, 0].cpu()[~bad].nan_to_num() - x[:, 0][~bad]).abs().max() <= 2.0 ** -4  # (1e-20 goes to 0; 1/6 in E4M3)


def test_cache_empty_calls_and_one_side():
    cache = nv.kv_cache(2, 2, 64, 16, device=DEV)
    none = torch.empty((0, 2, 64), device=DEV)
    nv.kv_write(none, none, cache, torch.empty(0, dtype=torch.int64, device=DEV))
    assert [t.shape for t in nv.kv_read(cache, torch.empty(0, dtype=torch.int64, device=DEV))] == [(0, 2, 64)] * 2
    x = torch.randn(5, 2, 64, device=DEV)
    slots = torch.arange(5, device=DEV) * 3
    nv.kv_write(x, -x, cache, slots)
    k, v = nv.kv_read(cache, slots)
    only = torch.empty_like(v)
    nv.nvfp4_kv_read(0, only.data_ptr(), nv.DTYPE_FP32, 5, 2, 64, slots.data_ptr(), cache.data_ptr(), 2, 16,
                     stream=torch.cuda.current_stream().cuda_stream)
    assert torch.equal(only, v) and torch.equal(k, -v)
    nothing = nv.kv_cache(0, 2, 64, 16, device=DEV)
    nv.kv_write(x, x, nothing, slots)
    assert not nv.kv_read(nothing, slots)[0].any()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def problem(rng, lens, counts, Hq, Hkv, D, page, dtype, encode=True, spread=1.0):
    """Random tokens in shuffled pages; unused places hold any bytes, NaN scales among them."""
    B = len(lens)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 2
    cache = rng.integers(0, 256, (pages, Hkv, page // 16, 2, D // 64, 576), dtype=np.uint8)
    cache[:, :, :, :, :, 512::3] = 0x7F
    table = rng.integers(-9, 99999, (B, max(used) + 1)).astype(np.int32)
    order = rng.permutation(pages)
    e = np.exp2(rng.integers(-1, 2, (2, Hkv))).astype(np.float32) if encode else (None, None)
    at = 0
    for b, n in enumerate(lens):
        table[b, : used[b]] = order[at: at + used[b]]
        at += used[b]
        k, v = rng.standard_normal((2, n, Hkv, D)).astype(np.float32)
        v += 0.25
        slots = np.array([int(table[b, t // page]) * page + t % page for t in range(n)], dtype=np.int64)
        write_fast(cache, slots, k * np.float32(spread), v, *e)
    T = sum(counts)
    q = torch.from_numpy(rng.standard_normal((T, Hq, D)).astype(np.float32)).to(DT[dtype])
    starts = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    return dict(cache=cache, table=table, lens=np.array(lens, dtype=np.int32), starts=starts, q=q, e=e, page=page)


def write_fast(cache, slots, k, v, e_k, e_v):
    """oa.write for whole arrays (the layout is tested there)."""
    from oracle import layer as ol

    page = cache.shape[2] * 16
    if len(slots) == 0:
        return
    for side, (x, e) in enumerate(((k, e_k), (v, e_v))):
        x = x if e is None else x * e[None, :, None]
        q, sf = ol.quantize(x)
        T, H = x.shape[:2]
        for c in range(cache.shape[4]):
            for h in range(H):
                rows = cache[slots // page, h, slots % page // 16, side, c]  # a copy
                i = np.arange(T)[:, None]
                rows[i, (slots % 16 * 32)[:, None] + np.arange(32)] = q[:, h, c * 32: c * 32 + 32]
                rows[i, (512 + slots % 16 * 4)[:, None] + np.arange(4)] = sf[:, h, c * 4: c * 4 + 4]
                for t in range(T):  # tokens share granules: each writes its own bytes
                    g = cache[slots[t] // page, h, slots[t] % page // 16, side, c]
                    a = slots[t] % 16
                    g[a * 32: a * 32 + 32] = rows[t, a * 32: a * 32 + 32]
                    g[512 + a * 4: 516 + a * 4] = rows[t, 512 + a * 4: 516 + a * 4]


def on_gpu(z):
    return dict(cache=gpu(z["cache"]), page_table=gpu(z["table"]), lengths=gpu(z["lens"]),
                encode_k=None if z["e"][0] is None else gpu(z["e"][0]),
                encode_v=None if z["e"][1] is None else gpu(z["e"][1]))


def check(z, out, lse, dtype, scale=None, **kw):
    q, page = z["q"].double().numpy(), z["page"]
    D = q.shape[2]
    kv, vv = oa.values(z["cache"])
    kv, vv = (x if e is None else x / e[:, None] for x, e in zip((kv, vv), z["e"]))
    got, got_lse = host(out), host(lse)
    for b, n in enumerate(z["lens"]):
        rows = slice(z["starts"][b], z["starts"][b + 1])
        slots = np.array([int(z["table"][b, t // page]) * page + t % page for t in range(n)], dtype=np.int64)
        want, want_lse, mix, bend = oa.attention(q[rows], kv[slots], vv[slots], scale or D ** -0.5, int(n), **kw)
        tol, tol_lse = oa.tolerance(want, mix, bend, int(n), D, HALF[dtype], np.abs(vv[slots]).max(initial=0))
        assert not np.isnan(got[rows]).any()
        worst = np.abs(got[rows] - want) - tol
        assert (worst <= 0).all(), (b, n, worst.max())
        empty = want_lse == -np.inf
        assert (got_lse[rows][empty] == -np.inf).all() and not got[rows][empty].any()
        assert (np.abs(got_lse[rows][~empty] - want_lse[~empty]) <= tol_lse[~empty]).all()


DECODE = [
    # lens, n, Hq, Hkv, D, page
    ([1], 1, 1, 1, 64, 16), ([2, 0, 31], 1, 4, 2, 128, 16), ([32, 33, 64, 65], 1, 8, 8, 64, 32),
    ([900], 1, 32, 8, 128, 64), ([17, 500, 3, 1201], 1, 24, 4, 256, 16), ([700, 5], 1, 7, 1, 128, 48),
    ([2500], 1, 16, 1, 128, 64), ([300, 100], 1, 40, 1, 64, 64), ([129, 257], 1, 33, 1, 128, 16),
    ([100, 50], 1, 71, 1, 256, 32), ([40, 41, 42], 3, 6, 2, 64, 16), ([600, 2, 70], 4, 16, 4, 128, 64),
    ([5, 1, 0], 7, 4, 4, 256, 16), ([333, 600], 9, 12, 3, 128, 128), ([150], 33, 5, 1, 64, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page", DECODE)
def test_attention(lens, n, Hq, Hkv, D, page, dtype):
    rng = np.random.default_rng(sum(lens) + Hq + D)
    z = problem(rng, lens, [n] * len(lens), Hq, Hkv, D, page, dtype)
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True)
    check(z, out, lse, dtype)
    again = nv.attention(z["q"].to(DEV), **on_gpu(z))
    assert torch.equal(out, again)


PROMPTS = [
    # more rows than the kernel for few query tokens takes: one, two and many row tiles, lengths
    # around the tiles' ends, queries without a prefix and behind one, rows before the sequence
    ([130], 130, 1, 1, 64, 16), ([300, 129], 128, 4, 2, 128, 64), ([70, 700], 65, 3, 3, 128, 48),
    ([513], 300, 8, 2, 64, 32), ([200, 128, 127], 100, 2, 1, 256, 16), ([256], 256, 6, 6, 256, 64),
    ([1030], 17, 40, 4, 128, 16), ([20, 0, 90], 80, 4, 4, 128, 16), ([1500], 3, 64, 1, 128, 64),
    # the row tiles are counted from above: one fewer than there is room for
    ([600], 64, 32, 8, 128, 64), ([400, 300], 64, 8, 1, 64, 16),
    # as many row tiles and heads as there are SMs and more: their tokens are not cut into parts
    ([140] * 10, 130, 16, 16, 64, 16), ([150, 131] * 6, 129, 14, 14, 128, 32), ([100, 90] * 8, 66, 12, 12, 256, 16),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,n,Hq,Hkv,D,page", PROMPTS)
def test_attention_of_prompts(lens, n, Hq, Hkv, D, page, dtype):
    rng = np.random.default_rng(sum(lens) + Hq + D)
    z = problem(rng, lens, [n] * len(lens), Hq, Hkv, D, page, dtype)
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True)
    check(z, out, lse, dtype)
    assert torch.equal(out, nv.attention(z["q"].to(DEV), **on_gpu(z)))


@pytest.mark.parametrize("window,causal,scale", [(1, True, None), (16, True, 0.3), (150, True, None), (0, False, None)])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(70, 8, 8, 64), (130, 4, 2, 128), (90, 3, 3, 256)])
def test_attention_of_prompts_masks(n, Hq, Hkv, D, window, causal, scale):
    rng = np.random.default_rng(window + n)
    z = problem(rng, [400, 131, 2, 140], [n] * 4, Hq, Hkv, D, 16, "fp16")
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True, window=window, causal=causal, scale=scale or 0.0)
    check(z, out, lse, "fp16", scale=scale, window=window, causal=causal)


def test_attention_of_prompts_and_single_tokens_together():
    """Both kernels in one call, sequences of no queries among them."""
    rng = np.random.default_rng(21)
    lens, counts = [900, 333, 64, 0, 512, 40, 700], [1, 200, 64, 0, 8, 33, 300]
    z = problem(rng, lens, counts, 8, 2, 128, 32, "bf16")
    out = torch.full((sum(counts) + 9, 8, 128), 3.0, dtype=torch.bfloat16, device=DEV)
    q = torch.cat((z["q"], torch.full((9, 8, 128), float("nan"), dtype=torch.bfloat16))).to(DEV)
    for max_q in (0, 300):
        out.fill_(3.0)
        _, lse = nv.attention(q, **on_gpu(z), q_starts=gpu(z["starts"]), max_q=max_q, return_lse=True, out=out)
        check(z, out[:-9], lse[:-9], "bf16")
        assert (out[-9:] == 3).all()
    # sequences with more query tokens than max_q says are left out, others are right
    right = out.clone()
    out.fill_(3.0)
    nv.attention(q, **on_gpu(z), q_starts=gpu(z["starts"]), max_q=8, out=out)
    few = torch.from_numpy(np.repeat([c <= 8 for c in counts] + [False], counts + [9])).to(DEV)
    assert torch.equal(out[few], right[few]) and (out[~few] == 3).all()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_of_prompts_does_not_see_masked_nan(D):
    rng = np.random.default_rng(22)
    z = problem(rng, [300], [140], 2, 2, D, 16, "fp16")
    full = z["cache"].copy()
    clean = nv.attention(z["q"].to(DEV), **on_gpu(z))
    for t in (299, 230, 161, 160, 100):
        page, at = int(z["table"][0, t // 16]), t % 16
        first = max(0, t - 160)  # the first query that sees the token
        z["cache"] = full.copy()
        z["cache"][page, 1, 0, 1, 0, 512 + at * 4 + 2] = 0x7F
        out = nv.attention(z["q"].to(DEV), **on_gpu(z))
        bad = torch.zeros(140, 2, D, dtype=torch.bool, device=DEV)
        bad[first:, 1, 32:48] = True
        assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad]), t
        z["cache"] = full.copy()
        z["cache"][page, 1, 0, 0, D // 64 - 1, 512 + at * 4] = 0x7F
        out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True)
        bad[:] = False
        bad[first:, 1] = True
        assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad]), t
        assert torch.equal(lse.isnan(), bad[..., 0])


def test_attention_of_prompts_pages_that_are_not_there():
    rng = np.random.default_rng(23)
    z = problem(rng, [300, 200], [140, 140], 2, 1, 128, 16, "bf16")
    good = nv.attention(z["q"].to(DEV), **on_gpu(z))
    for wrong in (-1, z["cache"].shape[0], 2 ** 31 - 1):
        t = z["table"].copy()
        t[0, 14] = wrong  # tokens 224 to 239: queries from 224 - 160 on
        out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z | {"table": t}), return_lse=True)
        assert out[64:140].isnan().all() and lse[64:140].isnan().all()
        assert torch.equal(out[:64], good[:64]) and torch.equal(out[140:], good[140:])
        t[0, 14], t[0, 1] = z["table"][0, 14], wrong
        assert nv.attention(z["q"].to(DEV), **on_gpu(z | {"table": t}))[:140].isnan().all()
    lens = np.array([z["table"].shape[1] * 16 + 1, 200], dtype=np.int32)
    table = np.where(np.arange(z["table"].shape[1]) < 13, z["table"], z["table"][1, 0])
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z | {"lens": lens, "table": np.abs(table) % z["cache"].shape[0]}),
                            return_lse=True)
    assert out[:140].isnan().all() and lse[:140].isnan().all()


@pytest.mark.parametrize("window,causal,scale", [(1, True, None), (16, True, 0.3), (33, True, None), (100, True, None),
                                                 (100000, True, None), (0, False, None), (0, False, 0.02)])
@pytest.mark.parametrize("n,Hq,Hkv,D", [(1, 8, 2, 128), (5, 6, 2, 64), (3, 4, 1, 256)])
def test_attention_masks(n, Hq, Hkv, D, window, causal, scale):
    rng = np.random.default_rng(window + n)
    z = problem(rng, [400, 31, 2, 97, 640], [n] * 5, Hq, Hkv, D, 16, "fp16")
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True, window=window, causal=causal, scale=scale or 0.0)
    check(z, out, lse, "fp16", scale=scale, window=window, causal=causal)


@pytest.mark.parametrize("max_q", [0, 40])
def test_attention_of_ragged_queries(max_q):
    rng = np.random.default_rng(11)
    lens, counts = [50, 7, 0, 300, 64, 33], [3, 0, 0, 40, 1, 33]
    z = problem(rng, lens, counts, 8, 4, 128, 32, "bf16")
    # rows in front of the first sequence and behind the last stay as they are
    q = torch.cat((torch.full((2, 8, 128), float("nan")), z["q"].float(), torch.full((5, 8, 128), float("nan")))).bfloat16()
    out = torch.full_like(q, 7.0, device=DEV)
    got, lse = nv.attention(q.to(DEV), **on_gpu(z), q_starts=gpu(z["starts"] + 2), max_q=max_q, return_lse=True, out=out)
    assert got is out
    T = sum(counts)
    check(z, out[2: T + 2], lse[2: T + 2], "bf16")
    assert (out[:2] == 7).all() and (out[T + 2:] == 7).all()


def test_attention_of_a_view_of_a_fused_row():
    rng = np.random.default_rng(12)
    z = problem(rng, [77, 130], [2, 2], 6, 3, 64, 16, "bf16")
    row = torch.full((4, 6 * 64 + 24), 3.0, dtype=torch.bfloat16, device=DEV)
    view = row[:, 8: 8 + 6 * 64].unflatten(1, (6, 64))
    view.copy_(z["q"])
    out, lse = nv.attention(view, **on_gpu(z), return_lse=True)
    check(z, out, lse, "bf16")
    by_head = z["q"].to(DEV).transpose(0, 1).contiguous().transpose(0, 1)  # heads far apart, tokens beside each other
    assert torch.equal(nv.attention(by_head, **on_gpu(z)), out)
    with pytest.raises(ValueError):
        nv.attention(row[:, 1: 1 + 6 * 64].unflatten(1, (6, 64)), **on_gpu(z))


def test_attention_does_not_see_masked_nan():
    """NaN scales in tokens that only later queries see, in K and in V."""
    rng = np.random.default_rng(13)
    z = problem(rng, [100], [6], 4, 2, 128, 16, "fp16")
    full = z["cache"].copy()
    page, at = int(z["table"][0, 97 // 16]), 97 % 16
    # V, token 97 (seen by the queries at 97, 98 and 99), elements 80..95 of head 1
    z["cache"][page, 1, 0, 1, 1, 512 + at * 4 + 1] = 0x7F
    out = nv.attention(z["q"].to(DEV), **on_gpu(z))
    clean = nv.attention(z["q"].to(DEV), **on_gpu(z | {"cache": full}))
    bad = torch.zeros(6, 4, 128, dtype=torch.bool, device=DEV)
    bad[3:, 2:, 80:96] = True
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad])
    # the same token in K: the whole rows
    z["cache"] = full.copy()
    z["cache"][page, 1, 0, 0, 1, 512 + at * 4 + 1] = 0xFF
    out = nv.attention(z["q"].to(DEV), **on_gpu(z))
    bad[:] = False
    bad[3:, 2:] = True
    assert torch.equal(out.isnan(), bad) and torch.equal(out[~bad], clean[~bad])
    # far from the end, where every query sees it
    z["cache"] = full.copy()
    z["cache"][int(z["table"][0, 2]), 0, 0, 1, 0, 512 + 5 * 4] = 0x7F
    out = nv.attention(z["q"].to(DEV), **on_gpu(z))
    bad[:] = False
    bad[:, :2, :16] = True
    assert torch.equal(out.isnan(), bad)


def test_attention_of_pages_that_are_not_there():
    """A page outside the cache makes NaN of the queries that see it, a length beyond the table of the
    sequence; nothing else changes."""
    rng = np.random.default_rng(14)
    z = problem(rng, [100, 60, 40], [2, 2, 2], 4, 2, 64, 16, "bf16")
    good, good_lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True)
    for wrong in (-1, z["cache"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = z["table"].copy()
        t[0, 6] = wrong  # tokens 96 to 99: both queries (98 and 99) see it
        t[1, 0] = wrong
        out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z | {"table": t}), return_lse=True)
        assert out[:4].isnan().all() and lse[:4].isnan().all()
        assert torch.equal(out[4:], good[4:]) and torch.equal(lse[4:], good_lse[4:])
        out = nv.attention(z["q"].to(DEV), **on_gpu(z | {"table": t}), window=30)
        assert out[:2].isnan().all() and not out[2:].isnan().any()  # (the second's page is out of sight)
    lens = np.array([z["table"].shape[1] * 16 + 1, 2 ** 31 - 1, 40], dtype=np.int32)
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z | {"lens": lens, "table": np.zeros_like(z["table"]) + z["table"][2:3]}),
                            return_lse=True)
    assert out[:4].isnan().all() and lse[:4].isnan().all() and torch.equal(out[4:], good[4:])
    lens = np.array([-5, 60, -2 ** 31], dtype=np.int32)
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z | {"lens": lens}), return_lse=True)
    assert not out[:2].any() and not out[4:].any() and torch.equal(out[2:4], good[2:4])
    assert (lse[:2] == -float("inf")).all()


def test_attention_of_large_and_small_queries():
    """bf16 values far outside fp16's range."""
    rng = np.random.default_rng(15)
    z = problem(rng, [70, 200], [1, 1], 4, 2, 64, 16, "bf16", encode=False)
    for size in (2.0 ** 60, 2.0 ** -60, 2.0 ** -126):
        z["q"] = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
        z["q"] = (z["q"].double() * size).bfloat16()
        scale = 0.125 / size if size < 2.0 ** 100 else 0.125
        if not 0 < np.float32(scale) < np.inf:
            scale = 0.125
        out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True, scale=float(np.float32(scale)))
        check(z, out, lse, "bf16", scale=float(np.float32(scale)))
    # scores that leave one token: the same result as that token's value
    z["q"] = z["q"].double().mul(2.0 ** 130).bfloat16()
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True)
    assert not out.isnan().any()


def test_attention_of_no_sequences():
    cache = nv.kv_cache(2, 2, 64, 16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = nv.attention(torch.empty((0, 4, 64), dtype=torch.float16, device=DEV), cache, torch.empty((0, 3), **i32),
                            torch.empty(0, **i32), return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    # no pages, and a table without any
    q = torch.randn(3, 4, 64, device=DEV).half()
    for table in (torch.zeros((3, 2), **i32), torch.empty((3, 0), **i32)):
        out, lse = nv.attention(q, nv.kv_cache(0, 2, 64, 16, device=DEV), table, torch.zeros(3, **i32), return_lse=True)
        assert not out.any() and (lse == -float("inf")).all()
    # no sequence has a query
    out = torch.full((3, 4, 64), 5.0, dtype=torch.float16, device=DEV)
    nv.attention(q, cache, torch.zeros((2, 2), **i32), torch.full((2,), 9, **i32), q_starts=torch.zeros(3, **i32), out=out)
    assert (out == 5).all()


def test_attention_of_many_sequences():
    """More sequences than a CTA has threads, most of them short, some without tokens."""
    rng = np.random.default_rng(16)
    lens = rng.integers(0, 40, 1300).tolist()
    z = problem(rng, lens, [1] * 1300, 2, 1, 64, 16, "fp16")
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), return_lse=True)
    check(z, out, lse, "fp16")


def test_attention_far_in_a_large_cache():
    """Pages beyond 2^32 bytes of the cache."""
    rng = np.random.default_rng(17)
    z = problem(rng, [300, 77], [1, 1], 16, 8, 128, 64, "bf16")
    few, page_bytes = z["cache"].shape[0], z["cache"][0].size
    pages = (1 << 32) // page_bytes + 2 * few
    if torch.cuda.mem_get_info()[0] < pages * page_bytes + (1 << 30):
        pytest.skip("needs 5 GB of free memory")
    big = torch.empty((pages, *z["cache"].shape[1:]), dtype=torch.uint8, device=DEV)
    big[pages - few:] = gpu(z["cache"])
    on = on_gpu(z)
    want = nv.attention(z["q"].to(DEV), **on)
    table = gpu(z["table"]) + (pages - few)
    assert torch.equal(nv.attention(z["q"].to(DEV), **(on | {"cache": big, "page_table": table})), want)
    # and the cache's own calls
    slots = torch.tensor([pages * 64 - 1, pages * 64 - 70, pages * 64], device=DEV)
    x = torch.randn(3, 8, 128, device=DEV)
    nv.kv_write(x, -x, big, slots)
    small = nv.kv_cache(2, 8, 128, 64, device=DEV)
    nv.kv_write(x, -x, small, slots - (pages - 2) * 64)
    assert torch.equal(big[pages - 2:], torch.where(small != 0, small, big[pages - 2:]))
    got, again = nv.kv_read(big, slots), nv.kv_read(small, slots - (pages - 2) * 64)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1]) and not got[0][2].any()
    del big
    torch.cuda.empty_cache()


def test_attention_replayed_from_a_graph_sees_new_lengths():
    """One captured step: rotate, write, attend; lengths, slots and positions change between replays."""
    rng = np.random.default_rng(18)
    B, Hq, Hkv, D, page = 3, 4, 2, 64, 16
    z = problem(rng, [40, 90, 7], [1] * B, Hq, Hkv, D, page, "bf16", encode=False)
    on = on_gpu(z)
    table = nv.rope_table(D)
    qkv = torch.randn(B, Hq + 2 * Hkv, D, device=DEV).bfloat16()
    positions = gpu(z["lens"]) - 1
    slots = torch.empty(B, dtype=torch.int64, device=DEV)
    work = torch.empty(nv.nvfp4_attention_workspace_bytes(B, B, Hq, Hkv, D, page, z["table"].shape[1]),
                       dtype=torch.uint8, device=DEV)
    out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV)
    turned = torch.empty(B, Hq + Hkv, D, dtype=torch.bfloat16, device=DEV)

    def place():
        p = positions.long()
        slots.copy_(on["page_table"].gather(1, (p // page).unsqueeze(1))[:, 0].long() * page + p % page)

    def step():
        nv.rope(qkv[:, : Hq + Hkv], positions, table, out=turned)
        nv.kv_write(turned[:, Hq:], qkv[:, Hq + Hkv:], on["cache"], slots)
        nv.attention(turned[:, :Hq], on["cache"], on["page_table"], on["lengths"], out=out, workspace=work)

    place()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        qkv.copy_(torch.randn(B, Hq + 2 * Hkv, D, device=DEV))
        if i and i != 3:  # the pages of problem() have room for two tokens more
            positions += 1
            on["lengths"] += 1
        place()
        out.fill_(float("nan"))
        graph.replay()
        got, cache = out.clone(), on["cache"].clone()
        step()
        assert torch.equal(got, out) and torch.equal(cache, on["cache"]) and not got.isnan().any()
        zz = z | {"cache": on["cache"].cpu().numpy(), "lens": on["lengths"].cpu().numpy(), "q": turned[:, :Hq].cpu()}
        _, lse = nv.attention(turned[:, :Hq], on["cache"], on["page_table"], on["lengths"], return_lse=True)
        check(zz, got, lse, "bf16")


def test_attention_calls_on_streams_at_once():
    """Calls that run side by side, with workspaces of their own, do not disturb each other."""
    rng = np.random.default_rng(19)
    zs = [problem(rng, [700 + 100 * i, 300], [1, 1], 16, 2, 128, 64, "bf16") for i in range(3)]
    ons = [on_gpu(z) for z in zs]
    qs = [z["q"].to(DEV) for z in zs]
    want = [nv.attention(q, **on) for q, on in zip(qs, ons)]
    streams = [torch.cuda.Stream() for _ in zs]
    torch.cuda.synchronize()
    for _ in range(20):
        got = [nv.attention(q, **on, stream=s) for q, on, s in zip(qs, ons, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_attention_of_a_long_sequence():
    """131,072 tokens: single tokens, passes of them, and rows for the prompt kernel."""
    rng = np.random.default_rng(30)
    z = problem(rng, [131072], [66], 2, 1, 64, 128, "bf16")
    for n in (66, 33, 1):
        zz = z | {"q": z["q"][-n:], "starts": np.array([0, n], dtype=np.int32)}
        out, lse = nv.attention(zz["q"].to(DEV), **on_gpu(zz), return_lse=True)
        check(zz, out, lse, "bf16")


def test_attention_of_many_ragged_sequences():
    """More sequences than the kernels' CTAs have threads, most without a query, a few with prompts."""
    rng = np.random.default_rng(31)
    B = 2300
    counts = (rng.random(B) < 0.3).astype(int)
    counts[[0, 1, 700, 1024, 2298, 2299]] = [70, 0, 129, 200, 65, 66]
    lens = (counts + rng.integers(0, 30, B)).tolist()
    z = problem(rng, lens, counts.tolist(), 1, 1, 64, 16, "bf16")
    out, lse = nv.attention(z["q"].to(DEV), **on_gpu(z), q_starts=gpu(z["starts"]), max_q=200, return_lse=True)
    check(z, out, lse, "bf16")


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 40), (256, 0)])
def test_attention_of_many_short_prompts(D, window):
    """More row tiles than CTAs are launched for: a CTA takes several, one after the other; NaN in the
    cache of some, and pages that do not exist, change those alone."""
    rng = np.random.default_rng(36)
    B = 700
    counts = rng.integers(20, 72, B)
    counts[rng.random(B) < 0.1] = 0
    lens = np.maximum(counts + rng.integers(-3, 60, B), 1)
    z = problem(rng, lens.tolist(), counts.tolist(), 4, 2, D, 16, "bf16")
    q, more = z["q"].to(DEV), dict(q_starts=gpu(z["starts"]), max_q=71, window=window, return_lse=True)
    out, lse = nv.attention(q, **on_gpu(z), **more)
    check(z, out, lse, "bf16", window=window)
    bad, nan = np.arange(3, B, 40), np.arange(7, B, 40)
    z["cache"][z["table"][nan, 0], :, 0, 0, 0, 512:] = 0x7F  # K
    z["cache"][z["table"][nan + 1, 0], :, 0, 1, 0, 512:] = 0xFF  # V
    z["table"][bad, 0] = -1
    got, got_lse = nv.attention(q, **on_gpu(z), **more)
    touched = np.isin(np.arange(B), np.concatenate((bad, nan, nan + 1)))
    rows = torch.from_numpy(np.repeat(touched, counts))
    assert torch.equal(got[~rows], out[~rows]) and torch.equal(got_lse[~rows], lse[~rows])
    assert torch.isnan(got[rows]).any()


def test_attention_with_starts_that_overlap():
    """Starts that are no partition of q's rows: no result is promised for the rows that are named
    twice or by a sequence that ends before it starts, every other row's is as it should be."""
    rng = np.random.default_rng(35)
    z = problem(rng, [300, 250, 200], [100, 90, 1], 4, 2, 64, 16, "bf16")
    q = z["q"].to(DEV)
    # the third sequence begins inside the first and ends at its own row; the fourth ends before it starts
    table = torch.cat((gpu(z["table"]), gpu(z["table"])[:1]))
    lens = torch.cat((gpu(z["lens"]), gpu(z["lens"])[:1]))
    on = on_gpu(z)
    want = nv.attention(q, **on, q_starts=gpu(z["starts"]), max_q=0)
    starts = torch.tensor([0, 100, 190, 150, 191], dtype=torch.int32, device=DEV)
    out = nv.attention(q, **(on | dict(page_table=table, lengths=lens)), q_starts=starts, max_q=0)
    assert torch.equal(out[:150], want[:150])


@pytest.mark.parametrize("n", [1, 80])
def test_attention_without_pages(n):
    """A cache and a page table without pages: empty sequences are 0, longer ones than the table NaN."""
    cache = nv.kv_cache(0, 2, 128, 16, device=DEV)
    q = torch.randn(2 * n, 4, 128, device=DEV).bfloat16()
    table = torch.zeros((2, 0), dtype=torch.int32, device=DEV)
    lengths = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    out, lse = nv.attention(q, cache, table, lengths, return_lse=True)
    assert not out[:n].any() and (lse[:n] == -float("inf")).all()
    assert torch.isnan(out[n:]).all() and torch.isnan(lse[n:]).all()
    assert nv.attention(q[:0], cache, table, lengths).shape == (0, 4, 128)


def test_attention_of_identical_pages():
    """Sequences that share pages (a common prefix) read the same tokens."""
    rng = np.random.default_rng(32)
    z = problem(rng, [96, 100], [1, 1], 4, 2, 128, 32, "bf16")
    z["table"][1, :3] = z["table"][0, :3]
    q = z["q"][:1].repeat(2, 1, 1)
    z = z | {"q": q, "lens": np.array([96, 96], dtype=np.int32)}
    out, lse = nv.attention(q.to(DEV), **on_gpu(z), return_lse=True)
    check(z, out, lse, "bf16")
    assert torch.equal(out[0], out[1]) and torch.equal(lse[0], lse[1])


LATE = 40_000_000  # clocks of a kernel that only waits, ~20 ms


@pytest.mark.parametrize("name", ["rope", "kv_write", "kv_read", "attention", "prompts"])
def test_calls_on_a_stream_given_by_name(name):
    """What a call allocates for another stream is neither still in use by the current one, nor handed
    out again while the call is to run."""
    rng = np.random.default_rng(33)
    n = 80 if name == "prompts" else 1
    z = problem(rng, [900, 700], [n, n], 8, 2, 128, 64, "bf16")
    on, q = on_gpu(z), z["q"].to(DEV)
    x = torch.randn(3000, 2, 128, device=DEV).bfloat16()
    slots = torch.arange(3000, device=DEV)
    other = nv.kv_cache(47, 2, 128, 64, device=DEV)
    pos, table = torch.arange(3000, dtype=torch.int32, device=DEV), nv.rope_table(128)
    call = {"rope": lambda s: [nv.rope(x, pos, table, stream=s)],
            "kv_write": lambda s: [nv.kv_write(x, x, other, slots, stream=s)],
            "kv_read": lambda s: list(nv.kv_read(other, slots, stream=s)),
            "attention": lambda s: list(nv.attention(q, **on, return_lse=True, stream=s)),
            "prompts": lambda s: list(nv.attention(q, **on, return_lse=True, stream=s))}[name]
    if name == "kv_read":
        nv.kv_write(x, -x, other, slots)
    want = [t.clone() for t in call(None)]
    other_bytes = other.clone()
    if name == "kv_write":
        other.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(LATE)
        got = call(side)  # runs late
        # the current stream allocates and fills memory meanwhile
        fills = [torch.full_like(t, 7) for t in got for _ in range(3)]
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all((f == 7).all() for f in fills)
        del got, fills
        torch.cuda.synchronize()
    if name == "kv_write":
        assert torch.equal(other, other_bytes)


def test_prompts_and_products_on_streams_at_once():
    """Kernels that take tensor memory side by side: attention of prompts and the quantised product."""
    rng = np.random.default_rng(34)
    zs = [problem(rng, [600], [150], 8, 2, D, 64, "bf16") for D in (64, 128, 256)]
    ons, qs = [on_gpu(z) for z in zs], [z["q"].to(DEV) for z in zs]
    a = torch.randn(1, 2048, 1024, device=DEV)
    w, sw = nv.quantize(a)
    rows = [nv.quantize(torch.randn(1, n, 1024, device=DEV)) for n in (5, 300, 2000)]
    calls = [lambda s, q=q, on=on: nv.attention(q, **on, stream=s) for q, on in zip(qs, ons)]
    calls += [lambda s, r=r: nv.gemm(w, r[0], sw, r[1], dtype=torch.float32, stream=s) for r in rows]
    want = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(15):
        got = [c(s) for c, s in zip(calls, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("steps", [0, 3])
def test_example_layer(steps):
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import attention_layer

    # bf16 outputs are off by at most 2^-8 of themselves, p by 2^-11
    assert attention_layer.main(steps) < 2.0 ** -7
