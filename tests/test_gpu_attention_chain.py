"""Rotation, cache and attention step after step through the same buffers: each call sees what the one before it wrote,
although its grid may have been launched before that one's end."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


@pytest.mark.parametrize("copied", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_steps_through_the_same_buffers(D, copied):
    """Ragged batches of prompts and single tokens with other starts in every step: the rotated rows, the cache's slots and
    the workspace (with its list of row tiles) are overwritten by each.  copied: starts, lengths and positions are
    copied into the same tensors too."""
    rng = np.random.default_rng(D)
    B, Hq, Hkv, page, steps, T = 5, 8, 2, 16, 12, 330
    pages = B * 20
    cache, table = nv.kv_cache(pages, Hkv, D, page, device=DEV), rng.permutation(pages).reshape(B, 20).astype(np.int32)
    qkv = [torch.randn(T, Hq + 2 * Hkv, D, device=DEV).bfloat16() for _ in range(steps)]
    plans = []
    for _ in range(steps):
        counts = rng.choice([0, 1, 1, 3, 40, 70, 150, 200], B)
        while counts.sum() > T:
            counts[rng.integers(B)] = 1
        lens = counts + rng.integers(0, 100, B)
        starts = np.concatenate(([0], np.cumsum(counts)))
        positions, slots = np.zeros(T, dtype=np.int32), np.full(T, -1, dtype=np.int64)
        for b in range(B):
            t = np.arange(lens[b] - counts[b], lens[b])
            positions[starts[b]: starts[b + 1]] = t
            slots[starts[b]: starts[b + 1]] = table[b, t // page] * page + t % page
        plans.append([gpu(x) for x in (starts.astype(np.int32), lens.astype(np.int32), positions, slots)])
    table, turns = gpu(table), nv.rope_table(D)
    turned = torch.empty(T, Hq + Hkv, D, dtype=torch.bfloat16, device=DEV)
    held = [torch.empty_like(x) for x in plans[0]]
    work = torch.empty(nv.nvfp4_attention_workspace_bytes(T, B, Hq, Hkv, D, page, 20, True, 0), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(T, Hq, D, dtype=torch.bfloat16, device=DEV) for _ in range(steps)]

    def run(after=lambda: None):
        for x, plan, out in zip(qkv, plans, outs):
            if copied:
                for h, p in zip(held, plan):
                    h.copy_(p)
                after()
            starts, lens, positions, slots = held if copied else plan
            nv.rope(x[:, : Hq + Hkv], positions, turns, out=turned)
            after()
            nv.kv_write(turned[:, Hq:], x[:, Hq + Hkv:], cache, slots)
            after()
            nv.attention(turned[:, :Hq], cache, table, lens, q_starts=starts, out=out, workspace=work)
            after()

    run(torch.cuda.synchronize)  # one call after the other
    want, after = [o.clone() for o in outs], cache.clone()
    assert not any(torch.equal(a, b) for a, b in zip(want, want[1:]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for again in range(6):
        for o in outs:
            o.zero_()
        cache.zero_()
        turned.zero_()
        work.fill_(255)
        torch.cuda.synchronize()
        # what a step finds beyond its own tokens is what the steps before wrote
        if again % 2:
            run()
        else:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), again
        assert torch.equal(cache, after)
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0
