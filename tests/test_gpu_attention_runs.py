"""Attention where a warp's run is many tiles and where a row tile's tokens are cut into parts: rings that go
round, references that rise again and again, pieces of items, parts with few or no tiles of their own."""
import functools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}
CTAS = 152


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0


@functools.lru_cache(maxsize=None)
def pool_of(D, Hkv, page, pages, rising):
    """Random pages.  rising: keys that grow from page to page, 16 times, 40-fold, and begin anew."""
    import attention64 as a64

    rng = np.random.default_rng(D + Hkv)
    k, v = rng.standard_normal((2, pages, page, Hkv, D)).astype(np.float32)
    if rising:
        k *= (40.0 ** (np.arange(pages) % 16 / 15)).astype(np.float32)[:, None, None, None]
    e = np.exp2(rng.integers(-1, 2, (2, Hkv))).astype(np.float32)
    cache = a64.pages_of(k.reshape(-1, Hkv, D), v.reshape(-1, Hkv, D) + np.float32(0.25), page, e)
    return a64.Pool(cache, page, e)


def tables(rng, lens, page, pages, wide=0):
    """Page numbers one after the other from anywhere in the pool, which sequences share."""
    most = max(max(-(-n // page) for n in lens), wide)
    return ((rng.integers(0, pages, (len(lens), 1)) + np.arange(most)) % pages).astype(np.int32)


# (D, query heads on a key head, query tokens): passes of 8, 16 and (heads of 64) 32 columns, and several of them
FEW = [(64, 4, 1), (64, 3, 5), (64, 8, 4), (64, 8, 8), (128, 4, 1), (128, 5, 3), (128, 8, 6), (256, 4, 1), (256, 4, 4),
       (256, 8, 5)]


@pytest.mark.parametrize("rising,window", [(False, 0), (True, 0), (True, 3000)])
@pytest.mark.parametrize("D,group,n", FEW)
def test_attention_of_long_runs(D, group, n, rising, window):
    """Every warp has at least 12 tiles one after the other (most of them 20 and more), which is several times
    round its ring; runs end inside items, and begin inside them."""
    import attention64 as a64

    rng = np.random.default_rng(D + group + n)
    Hkv, page, pages, B = 8, 64, 64, 48
    pool = pool_of(D, Hkv, page, pages, rising)
    lens = np.linspace(300, 16001, B).astype(int)
    if window:  # (fewer tiles each)
        lens = np.tile(lens, 2)
    rng.shuffle(lens)
    tile = 64 if D == 64 else 32
    tiles = sum(-(-min(x, window or x) // tile) for x in lens) * Hkv
    assert tiles >= 12 * 16 * CTAS
    table = tables(rng, lens, page, pages)
    q = torch.randn(len(lens) * n, Hkv * group, D, device=a64.DEV, generator=torch.Generator(a64.DEV).manual_seed(1))
    q = q.to(torch.bfloat16)
    call = dict(pool.call(), page_table=a64.gpu(table), lengths=a64.gpu(lens.astype(np.int32)), window=window)
    out, lse = nv.attention(q, **call, return_lse=True)
    passes = -(-n * group // 8)
    a64.check(pool, q, table, lens, [n] * len(lens), out, lse, tiles * passes * tile / (8 * CTAS) + 128, window=window)
    assert torch.equal(out, nv.attention(q, **call))


def parts(T, B, group, Hkv, D, ragged, max_q, room):
    """The parts that a row tile's tokens are cut into, by the rule of the kernels' host side."""
    few = 64 if D == 64 else 48
    most = (max_q if ragged else T // B) * group
    assert most > few
    pair = D == 256 and most > 128
    rows, tile, places = 128 if D == 256 and not pair else 256, 64 if D == 256 and not pair else 128, CTAS // (1 + pair)
    tiles = T * group // rows + min(T * group // (few + 1), B) if ragged else B * -(-T * group // B // rows)
    items = tiles * Hkv
    if items >= places:
        return 1
    fit = [s for s in range(1, 2 * places // max(items, 1) + 1) if s == 1 or s <= room // (4 * tile)]
    return min(fit, key=lambda s: (-(-s * items // places) / s + 0.01 * s, s))


# D, Hq, Hkv, (cached, query tokens) of the sequences, window, tokens that the page table has room for
PARTS = [
    # a chunk of a prompt far behind its beginning, with single tokens, an empty sequence and a short prompt
    (128, 8, 2, [(5000, 200), (900, 1), (40, 0), (2600, 70)], 0, 0),
    (128, 8, 2, [(5000, 200), (900, 1), (40, 0), (2600, 70)], 300, 0),
    (64, 6, 2, [(6000, 150), (100, 90), (3, 1)], 0, 0), (64, 6, 2, [(6000, 150), (100, 90)], 129, 0),
    # heads of 256 with up to 128 rows (one SM a row tile) and with more (a pair)
    (256, 4, 2, [(3000, 60), (50, 33), (700, 1)], 0, 0), (256, 4, 2, [(3000, 60), (2000, 33)], 100, 0),
    (256, 4, 2, [(4000, 200), (2500, 70), (9, 9)], 0, 0), (256, 4, 2, [(4000, 200), (2500, 70)], 500, 0),
    # as many tokens each
    (128, 4, 1, [(5000, 64), (130, 64)], 0, 0), (64, 8, 1, [(7000, 33), (33, 33)], 0, 0),
    (256, 8, 1, [(3000, 16), (90, 16)], 0, 0), (256, 8, 1, [(3000, 40), (41, 40)], 70, 0),
    # a table with room for far more than the sequences have: parts without a tile, queries before the sequence
    (128, 8, 1, [(512, 512)], 0, 65536), (128, 4, 2, [(130, 130), (20, 70)], 0, 8192),
    (64, 4, 2, [(130, 130), (20, 70), (0, 65)], 0, 8192), (256, 4, 2, [(64, 60), (20, 33)], 0, 8192),
    (256, 4, 2, [(130, 130), (20, 70)], 0, 8192), (256, 4, 2, [(600, 130), (600, 70)], 64, 16384),
    # fewer row tiles than could be: single tokens where there is room for prompts, and one prompt among them
    (128, 8, 2, [(700, 1)] * 90, 0, 4096), (64, 8, 2, [(700, 1)] * 90, 0, 4096), (256, 8, 2, [(700, 1)] * 90, 0, 4096),
    (128, 8, 2, [(700, 1)] * 40 + [(3000, 50)], 0, 4096), (64, 8, 2, [(700, 1)] * 40 + [(3000, 50)], 0, 4096),
    (256, 8, 2, [(700, 1)] * 40 + [(3000, 50)], 0, 4096),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("D,Hq,Hkv,sizes,window,room", PARTS)
def test_attention_of_row_tiles_in_parts(D, Hq, Hkv, sizes, window, room, dtype):
    import attention64 as a64

    rng = np.random.default_rng(D + len(sizes))
    page, pages = 32, 48
    pool = pool_of(D, Hkv, page, pages, False)
    lens, counts = (np.array(x) for x in zip(*sizes))
    table = tables(rng, lens, page, pages, room // page)
    T, starts = int(counts.sum()), np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    ragged = len(set(counts.tolist())) > 1 or counts[0] == 1
    max_q = int(counts.max()) if counts.max() > 1 else min(T, 60)
    assert parts(T, len(lens), Hq // Hkv, Hkv, D, ragged, max_q, table.shape[1] * page) > 1
    q = torch.randn(T, Hq, D, device=a64.DEV, generator=torch.Generator(a64.DEV).manual_seed(2)).to(DT[dtype])
    call = dict(pool.call(), page_table=a64.gpu(table), lengths=a64.gpu(lens.astype(np.int32)), window=window)
    if ragged:
        call |= dict(q_starts=a64.gpu(starts), max_q=max_q)
    out, lse = nv.attention(q, **call, return_lse=True)
    a64.check(pool, q, table, lens, counts, out, lse, [max(n, 1) for n in lens], window=window)
    assert torch.equal(out, nv.attention(q, **call))
    # a page that does not exist, in the middle: the rows that see it, and no others
    b, wrong = int(np.argmax(lens)), table.copy()
    at = (lens[b] - counts[b] // 2) // page
    wrong[b, at] = -1
    got, got_lse = nv.attention(q, **(call | dict(page_table=a64.gpu(wrong))), return_lse=True)
    j = np.arange(lens[b] - counts[b], lens[b])
    sees = (j >= at * page) & ((j - window < (at + 1) * page - 1) if window else True)
    rows = np.zeros(T, dtype=bool)
    rows[starts[b]: starts[b + 1]] = sees
    rows = torch.from_numpy(rows).to(a64.DEV)
    assert got[rows].isnan().all() and got_lse[rows].isnan().all()
    assert torch.equal(got[~rows], out[~rows]) and torch.equal(got_lse[~rows], lse[~rows])


LONG = [(1, 64), (32, 64), (16, 128), (8, 256), (66, 64), (60, 128), (40, 256), (120, 256)]


def long_call(q, pool, table, length):
    import attention64 as a64

    n, Hq, D = q.shape
    call = dict(pool.call(), page_table=a64.gpu(table), lengths=a64.gpu(np.array([length], dtype=np.int32)))
    # a run: a warp's tiles, or one of the ten parts that the host's rule cuts a row tile of this length into
    few = n * Hq <= (64 if D == 64 else 48)
    run = 2 * -(-n * Hq // 8) * length / (8 * CTAS) + 128 if few else length / 10
    return (*nv.attention(q, **call, return_lse=True), run, few)


@pytest.mark.parametrize("n,D", LONG)
def test_attention_of_a_long_sequence_adds_up_every_tile(n, D):
    """131,072 tokens of nearly equal weight: a tile of 32 is 2^-12 of their sum (the kernels for prompts have tiles
    of 64 or 128), and the sum may be off by less than half of a tile."""
    import attention64 as a64

    rng = np.random.default_rng(n)
    length, page, base = 131072, 128, 64
    k, v = rng.standard_normal((2, base * page, 1, D)).astype(np.float32)
    pool = a64.Pool(a64.pages_of(k / 16, v, page), page)
    table = rng.integers(0, base, (1, length // page)).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((n, 2, D)).astype(np.float32)).to(a64.DEV, torch.bfloat16)
    out, lse, run, few = long_call(q, pool, table, length)
    slots = a64.gpu(table[0, np.arange(length) // page].astype(np.int64) * page + np.arange(length) % page)
    r = a64.attend(q.double(), pool.k[slots], pool.v[slots], D ** -0.5, length)
    _, may = a64.bounds(r, D, 0.0, 1.0, run)
    tile = 32 if few and D > 64 else 64 if few or (D == 256 and 2 * n <= 128) else 128
    assert (2 * may < tile / length).all()
    a64.check(pool, q, table, [length], [n], out, lse, run)


@pytest.mark.parametrize("n,D", LONG)
def test_attention_of_a_long_sequence_finds_single_tokens(n, D):
    """131,072 tokens; each query and head has one that outweighs the others together, the first and last of tiles
    and pages all along, with a value of its own."""
    import attention64 as a64

    rng = np.random.default_rng(n)
    length, page, base, Hq = 131072, 128, 64, 2
    q = torch.from_numpy(rng.standard_normal((n, Hq, D)).astype(np.float32)).to(torch.bfloat16)
    k, v = (list(x) for x in rng.standard_normal((2, base, page, 1, D)).astype(np.float32))
    table = rng.integers(0, base, (1, length // page)).astype(np.int32)
    for i in range(n * Hq):
        t = {0: 0, n * Hq - 1: length - n}.get(i, (i + 1) * (length - n - 1) // (n * Hq) // 32 * 32 - i % 2)
        p = t // page
        if table[0, p] < base:  # (a page of its own)
            k.append(k[table[0, p]].copy())
            v.append(v[table[0, p]].copy())
            table[0, p] = len(k) - 1
        u, own = q[i // Hq, i % Hq].float().numpy(), table[0, p]
        k[own][t % page, 0] = u * np.float32(13.0 * D ** 0.5 / (u @ u))  # (a score of 13; the others' sum: e^12.3)
        v[own][t % page, 0] = rng.standard_normal(D) * 4
    pool = a64.Pool(a64.pages_of(np.concatenate(k), np.concatenate(v), page), page)
    q = q.to(a64.DEV)
    out, lse, run, _ = long_call(q, pool, table, length)
    a64.check(pool, q, table, [length], [n], out, lse, run)


@pytest.mark.parametrize("n", [1, 3, 70])
def test_attention_of_one_sequence_in_a_row_of_odd_length(n):
    """Views of a wider row: what a single token's row is followed by does not matter, nor a window beyond 32 bits."""
    import attention64 as a64

    pool = pool_of(128, 2, 32, 48, False)
    table = np.arange(40, dtype=np.int32)[None]
    wide = 8 * 128 + (3 if n == 1 else 8)
    row = torch.randn(n, wide, device=a64.DEV, generator=torch.Generator(a64.DEV).manual_seed(4)).bfloat16()
    q = row[:, : 8 * 128].unflatten(1, (8, 128))
    call = dict(pool.call(), page_table=a64.gpu(table), lengths=a64.gpu(np.array([1200], dtype=np.int32)))
    out, lse = nv.attention(q, **call, return_lse=True)
    a64.check(pool, q, table, [1200], [n], out, lse, 1200)
    assert torch.equal(out, nv.attention(q.contiguous(), **call))
    for window in (1 << 31, (1 << 32) + 5, 1 << 50):
        assert torch.equal(out, nv.attention(q, **call, window=window))
    assert not torch.equal(out, nv.attention(q, **call, window=5))


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_of_prompts_far_in_a_large_cache(D):
    """Pages beyond 2^32 bytes of the cache, and the places between them."""
    import attention64 as a64

    Hkv, page, pages = 2, 32, 48
    pool = pool_of(D, Hkv, page, pages, False)
    each = pool.cache[0].numel()
    far = (1 << 32) // each + 7
    if torch.cuda.mem_get_info()[0] < (far + pages) * each + (2 << 30):
        pytest.skip("needs 7 GB of free memory")
    big = torch.empty((far + pages, *pool.cache.shape[1:]), dtype=torch.uint8, device=a64.DEV)
    big[far:] = pool.cache
    rng = np.random.default_rng(D)
    lens, counts = np.array([1500, 300, 33]), np.array([90, 150, 1])
    table = tables(rng, lens, page, pages)
    q = torch.randn(int(counts.sum()), 4, D, device=a64.DEV, generator=torch.Generator(a64.DEV).manual_seed(5)).half()
    starts = a64.gpu(np.concatenate(([0], np.cumsum(counts))).astype(np.int32))
    call = dict(lengths=a64.gpu(lens.astype(np.int32)), q_starts=starts, max_q=150, encode_k=pool.e[0], encode_v=pool.e[1])
    want, lse = nv.attention(q, pool.cache, a64.gpu(table), **call, return_lse=True)
    a64.check(pool, q, table, lens, counts, want, lse, [1500] * 3)
    assert torch.equal(want, nv.attention(q, big, a64.gpu(table) + far, **call))
    del big
    torch.cuda.empty_cache()


# heads of 256: up to 128 rows of a sequence and key head (one SM a row tile), and more (a pair); in parts and whole
WIDE = [(2, 1, 66, [1131, 1162, 1345, 535, 334]), (2, 4, 17, [779, 545, 1534, 1597, 1566]), (8, 4, 17, [136, 512]),
        (3, 8, 9, [1149, 1830, 1438, 912, 131]), (1, 8, 66, [1079, 1771, 1749, 910, 459]), (2, 4, 130, [1500, 700]),
        (1, 1, 300, [1601]), (8, 4, 300, [1700, 300]), (8, 2, 60, [900] * 24)]


@pytest.mark.parametrize("window", [0, 1000])
@pytest.mark.parametrize("Hkv,group,n,lens", WIDE)
def test_attention_of_prompts_with_wide_heads_waits_for_its_last_products(Hkv, group, n, lens, window):
    """Few tiles a row tile, whose warps are then far apart: the results are read when the last product is through, call
    after call."""
    import attention64 as a64

    rng = np.random.default_rng(n + Hkv)
    page, pages = 32, 48
    pool = pool_of(256, Hkv, page, pages, False)
    lens = np.array(lens)
    table = tables(rng, lens, page, pages)
    q = torch.randn(n * len(lens), Hkv * group, 256, device=a64.DEV, generator=torch.Generator(a64.DEV).manual_seed(6)).half()
    call = dict(pool.call(), page_table=a64.gpu(table), lengths=a64.gpu(lens.astype(np.int32)), window=window)
    outs = [nv.attention(q, **call, return_lse=True) for _ in range(25)]
    for out, lse in outs:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    a64.check(pool, q, table, lens, [n] * len(lens), *outs[0], [int(x) for x in lens], window=window)
