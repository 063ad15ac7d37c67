"""The layer operators where a result can leave a type's range or be rounded once too often, on
the GPU, against formulas in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402
from oracle import layer as ol  # noqa: E402
from test_gpu_layer import DEV, DT, EPS, TINY, any_matrix, choices, gpu, host, values  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()
    yield
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0


# ---------------------------------------------------------------------------
# the experts' outputs before their sum
# ---------------------------------------------------------------------------

def experts(T, k, E, D, F, dtype, seed):
    """A layer's tensors, with alpha2 = 1."""
    rng = np.random.default_rng(seed)
    ids = choices(rng, T, k, E)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).to(DEV)
    w1, s1 = any_matrix(rng, E, 2 * F, D)
    w2, s2 = any_matrix(rng, E, D, F)
    a1 = np.full(E, 0.02 / np.sqrt(D), dtype=np.float32)
    return (x, gpu(ids), gpu(rng.random((T, k)).astype(np.float32)),
            [gpu(v) for v in (w1, ol.atoms(s1), w2, ol.atoms(s2))], gpu(a1))


def outputs(x, ids, m, a1, a2, dtype):
    """(the sort, the experts' rows of outputs as dtype) by the layer's steps."""
    order = nv.moe_sort(ids, m[0].shape[0])
    xq, xs = nv.quantize_rows(x, order)
    hq, hs = nv.moe_gated_gemm(m[0], m[1], xq, xs, order, alpha=a1, encode_scale=8.0)
    return order, nv.moe_gemm(m[2], m[3], hq, hs, order, alpha=a2, dtype=dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,k,E,D,F", [(40, 3, 5, 128, 64), (1500, 2, 7, 128, 64), (600, 8, 9, 160, 96)])
def test_experts_outputs_are_summed_before_they_are_rounded(T, k, E, D, F, dtype):
    """Outputs of 2e5 with weights below 0.01: beyond fp16 one by one, within it in their sum, and
    the sum is rounded once, for few choices and for many."""
    x, ids, w, m, a1 = experts(T, k, E, D, F, dtype, T)
    w = w * 0.01
    order, y = outputs(x, ids, m, a1, None, torch.float32)
    rows = order["rows"].long()
    a2 = torch.full((E,), 2e5, device=DEV) / y[rows].square().mean().sqrt()
    _, y = outputs(x, ids, m, a1, a2, torch.float32)
    terms = y[rows].double() * w.double().unsqueeze(-1)
    assert y[rows].abs().max() > 65504 and terms.abs().sum(1).max() < 65504
    out = nv.moe_ffn(x, ids, w, *m, alpha1=a1, alpha2=a2, encode_h=8.0)
    want = terms.sum(1)
    # fp32 sums of k terms, one rounding to the type
    tol = k * 2.0 ** -24 * terms.abs().sum(1) + EPS[dtype] * want.abs() + TINY[dtype]
    assert ((out.double() - want).abs() <= 1.01 * tol).all()
    assert torch.equal(out, nv.moe_combine(y, order, w, dtype=DT[dtype]))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,k", [(40, 3), (1500, 2)])
def test_experts_outputs_are_rounded_first_when_the_caller_says_so(T, k, dtype):
    x, ids, w, m, a1 = experts(T, k, 5, 128, 64, dtype, T + 1)
    order, y = outputs(x, ids, m, a1, a1, DT[dtype])
    out = nv.moe_ffn(x, ids, w, *m, alpha1=a1, alpha2=a1, encode_h=8.0, round_outputs=True)
    assert torch.equal(out, nv.moe_combine(y, order, w, dtype=DT[dtype]))
