"""Attention on scores far from zero, and on many tokens of small weight beside one of large."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402

pytestmark = pytest.mark.gpu
# query tokens (x 8 heads on one key head): passes of 8 and 16 columns, and the kernels for prompts
SHAPES = [(1, 64), (4, 64), (100, 64), (1, 128), (2, 128), (100, 128), (1, 256), (2, 256), (15, 256), (100, 256)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()


@pytest.fixture(autouse=True)
def _no_timeouts():
    yield
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0


def random_pool(rng, tokens, D):
    import attention64 as a64

    k, v = rng.standard_normal((2, tokens, 1, D)).astype(np.float32)
    return a64.Pool(a64.pages_of(k, v, 64), 64)


@pytest.mark.parametrize("n,D", SHAPES)
@pytest.mark.parametrize("e", [4, 12, 18, 20, 22, 24, 26, 28, 31, 40, 60])
def test_attention_of_scores_far_from_zero(n, D, e):
    """Queries of size 2^e: one token has all the weight, wherever its score lies more above the second's than
    scores may be off by, and is the result; lse is its score.  No row is NaN or without weight."""
    import attention64 as a64

    rng = np.random.default_rng(e)
    length = 900
    pool = random_pool(rng, 960, D)
    q = torch.from_numpy(rng.standard_normal((n, 8, D)) * 2.0 ** e).to(a64.DEV, torch.bfloat16)
    table, lengths = torch.arange(15, dtype=torch.int32, device=a64.DEV)[None], torch.full((1,), length, dtype=torch.int32, device=a64.DEV)
    out, lse = nv.attention(q, **pool.call(), page_table=table, lengths=lengths, return_lse=True)
    r = a64.attend(q.double(), pool.k[:length], pool.v[:length], D ** -0.5, length)
    # a score is an fp32 sum of D products in D/16 steps that may each lose 2^-22 of what is summed, and four more
    # roundings of its size: off by d at most
    d = r["bend"] * (D / 16 + 4) * 2.0 ** -22
    sure = r["gap"] > 2 * d + 30
    assert e < 12 or sure.double().mean() >= 0.75  # (of the inputs alone: most rows are compared)
    assert not out.isnan().any() and not lse.isnan().any()
    assert ((lse.double() - r["lse"]).abs() <= d + 2.0 ** -22 * r["bend"] + 2.0 ** -11)[sure].all()
    want = pool.v[:length, 0][r["top"].long()]
    # (e^-30 of other tokens; bf16's half step)
    assert ((out.double() - want).abs() <= 2.0 ** -8 * want.abs() * (1 + 2.0 ** -6) + length * math.exp(-30) * 16)[sure].all()
    # rows with more than one token in question hold something between the tokens' values
    low, high = pool.v[:length, 0].amin(0), pool.v[:length, 0].amax(0)
    assert ((out.double() >= low - 2.0 ** -7 * low.abs()) & (out.double() <= high + 2.0 ** -7 * high.abs())).all()


@pytest.mark.parametrize("gap", [8, 14, 16, 17, 18])
@pytest.mark.parametrize("n,D", SHAPES)
def test_attention_of_many_tokens_of_small_weight(n, D, gap):
    """The first token, whose value is 0, outweighs each of the 131,071 others by e^gap: what is left of the result
    is the others', each of which has a weight far below 2^-14."""
    import attention64 as a64

    rng = np.random.default_rng(gap)
    page, base, length = 128, 33, 131072
    k, v = np.zeros((base * page, 1, D), dtype=np.float32), rng.standard_normal((base * page, 1, D)).astype(np.float32) + 3
    k[:, 0, 0] = -gap / 2
    k[0, 0, 0] = gap / 2
    v[0] = 0
    pool = a64.Pool(a64.pages_of(k, v, page), page)
    table = rng.integers(1, base, (1, length // page)).astype(np.int32)
    table[0, 0] = 0
    q = torch.zeros(n, 8, D, dtype=torch.bfloat16, device=a64.DEV)
    q[..., 0] = 1
    call = dict(pool.call(), page_table=a64.gpu(table), lengths=a64.gpu(np.array([length], dtype=np.int32)), scale=1.0)
    out, lse = nv.attention(q, **call, return_lse=True)
    few = n * 8 <= (64 if D == 64 else 48)
    run = 2 * n * length / (8 * 152) + 128 if few else length / 10
    a64.check(pool, q, table, [length], [n], out, lse, run, scale=1.0)
