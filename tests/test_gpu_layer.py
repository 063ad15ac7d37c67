"""The layer operators on the GPU against the 64-bit oracle.

Integers keep the products exact: E2M1 codes of whole values and power-of-two
scales make every partial sum a whole number below 2^24, so any order of an
fp32 sum gives the same result and the comparison is for equality.  General
values are held to the library's accuracy contract, 1e-3 * sum|terms| plus the
rounding to the output type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402
from oracle import layer as ol  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TINY = {"fp16": 2.0 ** -24, "bf16": 2.0 ** -126, "fp32": 2.0 ** -126}  # a unit of the smallest results


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()
    yield
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def host(t):
    return t.cpu().numpy()


def values(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# quantise
# ---------------------------------------------------------------------------

def rows_of(rng, rows, K, dtype):
    """Values of many magnitudes, with ties of both formats among them."""
    x = rng.standard_normal((rows, K)) * np.exp(rng.standard_normal((rows, 1)))
    x[rng.random(x.shape) < 0.02] = 0
    n = rows * (K // 16)
    blocks = x.reshape(n, 16)
    # blocks of whole multiples of a scale: exact ties of the codes
    at = rng.random(n) < 0.3
    s = ol.e4m3_values(rng.integers(8, 0x70, n).astype(np.uint8))
    ties = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], (n, 16)) * rng.choice([-1, 1], (n, 16))
    ties[:, 0] = 6.0
    blocks[at] = (ties * s[:, None])[at]
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype])


@pytest.mark.parametrize("layout", [nv.SF_PLAIN, nv.SF_PERMUTED_128x4])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,K,encode", [(1, 16, 1.0), (1, 4096, 0.7), (3, 80, 1.0), (129, 208, 3.3),
                                           (128, 64, 1.0), (257, 1024, 0.011), (40, 8192, 1.0),
                                           (2500, 8272, 1.7)])
def test_quantize_bit_exact(rows, K, encode, dtype, layout):
    rng = np.random.default_rng(rows * 7 + K)
    x = rows_of(rng, rows, K, dtype)
    q, sf = nv.quantize(x.to(DEV), encode_scale=encode, sf_layout=layout)
    want_q, want_sf = ol.quantize(x.float().numpy(), encode)
    if layout == nv.SF_PERMUTED_128x4:
        assert np.array_equal(host(sf), ol.atoms(want_sf[None]))
    else:
        assert np.array_equal(host(sf), want_sf.reshape(-1))
    assert np.array_equal(host(q), want_q)


def test_quantize_every_scale_with_every_tie():
    """For each scale s: a block whose largest is 6 s, all ties of the codes, and their
    neighbours in fp32; and the ties between scales, with theirs."""
    s = ol.e4m3_values(np.arange(1, 0x7F, dtype=np.uint8)).astype(np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    blocks = []
    for toward in (None, np.float32(0), np.float32(1e9)):
        t = ties[None] * s[:, None]
        t = t if toward is None else np.nextafter(t, toward)
        blocks.append(np.concatenate((6 * s[:, None], t, -t, np.zeros((len(s), 1), np.float32)), axis=1))
    mid = 6 * (s[1:] + s[:-1]) / 2
    for toward in (mid, np.float32(0), np.float32(1e9)):
        b = np.zeros((len(mid), 16), dtype=np.float32)
        b[:, 3], b[:, 5] = np.nextafter(mid, toward), 0.3 * mid
        blocks.append(b)
    x = np.concatenate(blocks).reshape(-1, 16)
    x = np.concatenate((x, np.zeros((-len(x) % 4, 16), np.float32))).reshape(-1, 64)
    q, sf = nv.quantize(gpu(x), sf_layout=nv.SF_PLAIN)
    want_q, want_sf = ol.quantize(x)
    assert np.array_equal(host(sf), want_sf.reshape(-1))
    assert np.array_equal(ol.e2m1_values(host(q)), ol.e2m1_values(want_q))


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_quantize_strided_and_unaligned_rows(dtype):
    rng = np.random.default_rng(5)
    wide = rows_of(rng, 37, 160, dtype).to(DEV)
    for lo, K in ((0, 128), (8, 128), (1, 96), (3, 16)):
        x = wide[:, lo:lo + K]
        q, sf = nv.quantize(x, sf_layout=nv.SF_PLAIN)
        want_q, want_sf = ol.quantize(x.float().cpu().numpy())
        assert np.array_equal(host(q), want_q) and np.array_equal(host(sf), want_sf.reshape(-1))


def test_quantize_batches():
    rng = np.random.default_rng(6)
    x = rows_of(rng, 3 * 130, 96, "bf16").view(3, 130, 96)
    q, sf = nv.quantize(x.to(DEV))
    want_q, want_sf = ol.quantize(x.float().numpy())
    assert np.array_equal(host(q), want_q) and np.array_equal(host(sf), ol.atoms(want_sf))


def test_quantize_special_values():
    x = np.zeros((8, 32), dtype=np.float32)
    x[0] = -0.0
    x[1, 3] = np.nan
    x[2, 20] = -np.inf
    x[3] = 3e38             # finite, times 4 is not
    x[4] = 1e-42            # subnormal
    x[5, :16], x[5, 16:] = 1e6, -1e6  # saturates the scale and the codes
    x[6, 0] = 6 * 2.0 ** -10           # a tie between a zero scale and the smallest: to zero
    x[7, 0] = np.nextafter(np.float32(6 * 2.0 ** -10), np.float32(1))
    for encode in (1.0, 4.0):
        q, sf = nv.quantize(gpu(x), encode_scale=encode, sf_layout=nv.SF_PLAIN)
        want_q, want_sf = ol.quantize(x, encode)
        assert np.array_equal(host(sf).reshape(8, 2), want_sf)
        got, want = ol.e2m1_values(host(q)), ol.e2m1_values(want_q)
        assert np.array_equal(got, want)
    assert np.isnan(values(nv.dequantize(*nv.quantize(gpu(x)), dtype=torch.float32))[1, :16]).all()


@pytest.mark.parametrize("layout", [nv.SF_PLAIN, nv.SF_PERMUTED_128x4])
def test_quantize_into_named_rows(layout):
    rng = np.random.default_rng(8)
    rows, K, cap = 19, 208, 300
    x = rows_of(rng, rows, K, "bf16")
    to = rng.permutation(cap)[:rows * 3].reshape(rows, 3).astype(np.int32)
    to[2, 1], to[5, 0], to[6, 2] = -1, cap, -7  # skipped
    q = torch.full((cap, K // 2), 0xA5, dtype=torch.uint8, device=DEV)
    sf = torch.full((nv.nvfp4_permuted_scale_bytes(cap, K, 1) if layout else cap * (K // 16),), 0xA5,
                    dtype=torch.uint8, device=DEV)
    xd, td = x.to(DEV), gpu(to)
    nv.nvfp4_quantize(xd.data_ptr(), nv.DTYPE_BF16, rows, K, 1, q.data_ptr(), sf.data_ptr(), layout, 1.0,
                      row_map=td.data_ptr(), copies=3, q_rows=cap,
                      stream=torch.cuda.current_stream().cuda_stream)
    want_q, want_sf = ol.quantize(x.float().numpy())
    full_q = np.full((cap, K // 2), 0xA5, dtype=np.uint8)
    full_sf = np.full((cap, K // 16), 0xA5, dtype=np.uint8)
    for r in range(rows):
        for d in to[r]:
            if 0 <= d < cap:
                full_q[d], full_sf[d] = want_q[r], want_sf[r]
    assert np.array_equal(host(q), full_q)
    if layout == nv.SF_PLAIN:
        assert np.array_equal(host(sf).reshape(cap, -1), full_sf)
    else:
        # K % 64 != 0: the padding blocks of a written row are zero, of the others untouched
        full = ol.from_atoms(host(sf), 384, 16)[0]
        named = sorted(int(d) for d in to.ravel() if 0 <= d < cap)
        assert np.array_equal(full[:cap, :13], full_sf)
        assert not full[named, 13:].any()
        others = np.setdiff1d(np.arange(384), named)
        assert (full[others] == 0xA5).all()


@pytest.mark.parametrize("layout", [nv.SF_PLAIN, nv.SF_PERMUTED_128x4])
@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
def test_dequantize_all_codes(dtype, layout):
    """Every code with every scale code, and a scale: one rounding after an exact product."""
    rows, K = 130, 256 * 16
    q = np.tile(np.arange(256, dtype=np.uint8), (rows, K // 512))
    sf = np.broadcast_to(np.arange(256, dtype=np.uint8), (rows, 256)).copy()
    flat = ol.atoms(sf[None]) if layout else sf.reshape(-1)
    for scale in (1.0, 0.3):
        x = nv.dequantize(gpu(q), gpu(flat), scale=scale, dtype=DT[dtype], sf_layout=layout)
        want = torch.from_numpy(ol.matrix(q, sf)).float() * torch.tensor(scale, dtype=torch.float32)
        assert torch.equal(torch.nan_to_num(x.cpu().float(), nan=1e9),
                           torch.nan_to_num(want.to(DT[dtype]).float(), nan=1e9))


@pytest.mark.parametrize("layout", [nv.SF_PLAIN, nv.SF_PERMUTED_128x4])
@pytest.mark.parametrize("stride,offset", [(96, 0), (104, 0), (97, 1), (2080, 16)])
def test_dequantize_batches_into_strided_rows(stride, offset, layout):
    rng = np.random.default_rng(stride)
    L, rows, K = 2, 131, 2064 if stride > 2000 else 96
    q = rng.integers(0, 256, (L, rows, K // 2), dtype=np.uint8)
    sf = rng.integers(0, 0x7F, (L, rows, K // 16)).astype(np.uint8)
    buf = torch.full((L * rows * stride + offset,), -77.0, dtype=torch.float16, device=DEV)
    qd, sd = gpu(q), gpu(ol.atoms(sf) if layout else sf.reshape(-1))
    nv.nvfp4_dequantize(qd.data_ptr(), sd.data_ptr(), rows, K, L, buf.data_ptr() + 2 * offset, nv.DTYPE_FP16,
                        layout, x_row_stride=stride, stream=torch.cuda.current_stream().cuda_stream)
    got = values(buf)
    assert (got[:offset] == -77).all()
    got = got[offset:].reshape(L, rows, stride)
    assert np.array_equal(got[:, :, :K], ol.matrix(q, sf)) and (got[:, :, K:] == -77).all()


@pytest.mark.parametrize("layout", [nv.SF_PLAIN, nv.SF_PERMUTED_128x4])
def test_fold_scale_signs_keeps_the_values(layout):
    rng = np.random.default_rng(9)
    L, rows, K = 2, 131, 80
    a = rng.integers(0, 256, (L, rows, K // 2), dtype=np.uint8)
    sf = rng.integers(0, 256, (L, rows, K // 16), dtype=np.uint8)
    flat = ol.atoms(sf) if layout else sf.reshape(-1)
    ad, sd = nv.fold_scale_signs(gpu(a), gpu(flat), layout)
    new = ol.from_atoms(host(sd), rows, K // 16, L) if layout else host(sd).reshape(sf.shape)
    assert np.array_equal(new, sf & 0x7F)
    assert np.array_equal(ol.matrix(host(ad), new), ol.matrix(a, sf), equal_nan=True)


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

WHOLE = np.array([0, 2, 4, 5, 6, 8, 10, 12, 13, 14], dtype=np.uint8)  # codes of 0, 1, 2, 3, 4 and their negatives


def whole_matrix(rng, *shape):
    """Codes [..., K/2] of whole values and scales [..., K/16] of 1 or 2."""
    lo, hi = rng.choice(WHOLE, (*shape[:-1], shape[-1] // 2)), rng.choice(WHOLE, (*shape[:-1], shape[-1] // 2))
    return (lo | (hi << 4)).astype(np.uint8), rng.choice(np.array([0x38, 0x40], dtype=np.uint8),
                                                         (*shape[:-1], shape[-1] // 16))


def any_matrix(rng, *shape):
    return (rng.integers(0, 256, (*shape[:-1], shape[-1] // 2), dtype=np.uint8),
            rng.integers(0x20, 0x50, (*shape[:-1], shape[-1] // 16)).astype(np.uint8))


def run_gemm(a, sfa, b, sfb, **kw):
    return nv.gemm(gpu(a), gpu(b), gpu(ol.atoms(sfa)), gpu(ol.atoms(sfb)), **kw)


@pytest.mark.parametrize("M,K,L", [(1, 32, 1), (128, 256, 1), (131, 64, 2), (300, 1056, 1), (513, 2080, 2)])
@pytest.mark.parametrize("N", [1, 2, 16, 17, 31, 33, 64, 65, 127, 128, 129, 256, 257, 385, 600])
def test_gemm_exact_on_whole_numbers(N, M, K, L):
    rng = np.random.default_rng(N * 1000 + M + K)
    a, sfa = whole_matrix(rng, L, M, K)
    b, sfb = whole_matrix(rng, L, N, K)
    want, _ = ol.gemm(ol.matrix(a, sfa), ol.matrix(b, sfb))
    c = run_gemm(a, sfa, b, sfb, dtype=torch.float32)
    assert np.array_equal(values(c), want)


def test_gemm_exact_larger():
    """More tiles than CTAs, every N tile, odd sizes: the persistent loop and its rings."""
    rng = np.random.default_rng(77)
    for N, M, K, L in ((24, 5000, 4128, 2), (100, 7000, 2048, 1), (700, 4100, 1120, 2), (1025, 3001, 416, 3)):
        a, sfa = whole_matrix(rng, L, M, K)
        b, sfb = whole_matrix(rng, L, N, K)
        got = run_gemm(a, sfa, b, sfb, dtype=torch.float32)
        at, bt = (torch.from_numpy(ol.matrix(*m)).to(DEV).float() for m in ((a, sfa), (b, sfb)))
        # whole numbers below 2^24: fp32 products on the GPU are exact in any order
        assert torch.equal(got, torch.bmm(bt, at.transpose(1, 2)))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("N,M,K,L", [(2300, 4100, 2080, 1), (2304, 4096, 2048, 1), (2300, 4101, 2080, 1),
                                     (1153, 4224, 4096, 2), (385, 20000, 8192, 1), (449, 20000, 8192, 1),
                                     (256 + 64, 20000, 8192, 1), (256 + 180, 20000, 8224, 1)])
def test_gemm_exact_on_pairs_of_sms(N, M, K, L, dtype):
    """256-row tiles: more tiles than pairs, both accumulators, narrow last tiles, rows of c
    that TMA can store and rows that it cannot."""
    assert nv.nvfp4_gemm_plan(M, N, K, L, torch.cuda.get_device_properties(0).multi_processor_count) == {
        "tile_rows": 256, "k_split": 1}
    rng = np.random.default_rng(N + M)
    a, sfa = whole_matrix(rng, L, M, K)
    b, sfb = whole_matrix(rng, L, N, K)
    got = run_gemm(a, sfa, b, sfb, alpha=2.0 ** -6, dtype=DT[dtype])
    at, bt = (torch.from_numpy(ol.matrix(*m)).float().to(DEV) for m in ((a, sfa), (b, sfb)))
    # whole numbers below 2^24 times a power of two: exact in fp32, one rounding to the type
    assert torch.equal(got, (torch.bmm(bt, at.transpose(1, 2)) * 2.0 ** -6).to(DT[dtype]))


@pytest.mark.parametrize("N,M,K,L,split", [(1, 513, 2080, 1, 2), (16, 4096, 4096, 1, 4), (30, 2048, 4128, 2, 4),
                                           (40, 1000, 8192, 1, 2), (100, 1000, 8192, 1, 2), (7, 640, 4096, 3, 4)])
def test_gemm_exact_with_split_k(N, M, K, L, split):
    plan = nv.nvfp4_gemm_plan(M, N, K, L, torch.cuda.get_device_properties(0).multi_processor_count)
    assert plan["k_split"] == split
    rng = np.random.default_rng(N + M)
    a, sfa = whole_matrix(rng, L, M, K)
    b, sfb = whole_matrix(rng, L, N, K)
    want, _ = ol.gemm(ol.matrix(a, sfa), ol.matrix(b, sfb))
    for _ in range(3):
        assert np.array_equal(values(run_gemm(a, sfa, b, sfb, dtype=torch.float32)), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("act", range(5))
def test_gemm_general_values_and_epilogue(act, dtype):
    rng = np.random.default_rng(act)
    for N, M, K, L in ((5, 200, 544, 2), (150, 130, 288, 1)):
        a, sfa = any_matrix(rng, L, M, K)
        b, sfb = any_matrix(rng, L, N, K)
        bias = rng.standard_normal((L, M)).astype(np.float32)
        alpha = 0.01
        want, sums = ol.gemm(ol.matrix(a, sfa), ol.matrix(b, sfb), np.float32(alpha), bias, act)
        c = run_gemm(a, sfa, b, sfb, alpha=alpha, bias=gpu(bias), activation=act, dtype=DT[dtype])
        # 1.13 bounds every activation's slope; a few fp32 ulps of its evaluation
        tol = 1.13 * 1e-3 * sums + (EPS[dtype] + 8 * EPS["fp32"]) * np.abs(want) + 1e-6 + TINY[dtype]
        assert (np.abs(values(c) - want) <= tol).all()


def test_gemm_row_stride_leaves_the_gap():
    rng = np.random.default_rng(3)
    M, N, K = 70, 20, 96
    a, sfa = whole_matrix(rng, 1, M, K)
    b, sfb = whole_matrix(rng, 1, N, K)
    c = torch.full((N, M + 9), -77.0, dtype=torch.float32, device=DEV)
    t = [gpu(a), gpu(b), gpu(ol.atoms(sfa)), gpu(ol.atoms(sfb))]
    nv.nvfp4_gemm(*[x.data_ptr() for x in t], c.data_ptr(), M, N, K, 1, c_dtype=nv.DTYPE_FP32,
                  c_row_stride=M + 9, stream=torch.cuda.current_stream().cuda_stream)
    want, _ = ol.gemm(ol.matrix(a, sfa), ol.matrix(b, sfb))
    assert np.array_equal(values(c)[:, :M], want[0]) and (values(c)[:, M:] == -77).all()


def test_gemm_without_k():
    bias = torch.randn(2, 50, device=DEV)
    e = torch.empty(0, dtype=torch.uint8, device=DEV)
    c = nv.gemm(e.view(2, 50, 0), e.view(2, 7, 0), e, e, bias=bias, activation=nv.ACT_RELU, dtype=torch.float32)
    assert torch.equal(c, bias.relu().unsqueeze(1).expand(2, 7, 50))
    c = nv.gemm(e.view(2, 50, 0), e.view(2, 7, 0), e, e, dtype=torch.float32)
    assert torch.equal(c, torch.zeros(2, 7, 50, device=DEV))


def test_gemm_nan_scales_and_signs():
    rng = np.random.default_rng(4)
    M, N, K = 140, 40, 128
    a, sfa = whole_matrix(rng, 1, M, K)
    b, sfb = whole_matrix(rng, 1, N, K)
    b[:], sfb[0, 7, 3] = np.where(b == 0, 0x22, b), 0x7F
    sfa[0, 131, 2] = 0x7F
    c = values(run_gemm(a, sfa, b, sfb, dtype=torch.float32))[0]
    nan = np.zeros((N, M), dtype=bool)
    nan[7], nan[:, 131] = True, True
    assert np.array_equal(np.isnan(c), nan)
    # bit 7 of a scale is ignored; folding it first gives the signed product
    sfa, sfb = sfa & 0x47, sfb & 0x47
    signed = sfa | (rng.integers(0, 2, sfa.shape) << 7).astype(np.uint8)
    assert np.array_equal(values(run_gemm(a, signed, b, sfb, dtype=torch.float32)),
                          ol.gemm(ol.matrix(a, sfa), ol.matrix(b, sfb))[0])
    ad, sd = nv.fold_scale_signs(gpu(a), gpu(ol.atoms(signed)))
    c = nv.gemm(ad, gpu(b), sd, gpu(ol.atoms(sfb)), dtype=torch.float32)
    assert np.array_equal(values(c), ol.gemm(ol.matrix(a, signed), ol.matrix(b, sfb))[0])


def test_gemm_repeats_bit_for_bit_on_another_stream():
    rng = np.random.default_rng(5)
    a, sfa = any_matrix(rng, 1, 700, 1024)
    b, sfb = any_matrix(rng, 1, 300, 1024)
    t = [gpu(a), gpu(b), gpu(ol.atoms(sfa)), gpu(ol.atoms(sfb))]
    first = nv.gemm(*t, dtype=torch.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        outs = [nv.gemm(*t, dtype=torch.float32) for _ in range(5)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


def test_quantized_product_in_a_graph():
    """quantise -> product, captured and replayed on new inputs."""
    rng = np.random.default_rng(6)
    M, N, K = 260, 40, 288
    a, sfa = whole_matrix(rng, 1, M, K)
    ad, sd = gpu(a), gpu(ol.atoms(sfa))
    x = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)

    def step():
        q, sf = nv.quantize(x)
        return nv.gemm(ad, q.unsqueeze(0), sd, sf, dtype=torch.float32)

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c = step()
    for i in range(3):
        # whole numbers up to 6 with a 6 in every block: the quantisation is exact
        v = rng.choice([0, 1, 2, 3, 4, 6], (N, K)) * rng.choice([-1, 1], (N, K))
        v[:, ::16] = 6
        x.copy_(torch.from_numpy(v))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(values(c)[0], v.astype(float) @ ol.matrix(a, sfa)[0].T)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def logits_of(rng, T, E, dtype, levels=None):
    """Logits on a grid of 1/16 (exact in every type), so that equal ones tie exactly."""
    return torch.from_numpy(rng.integers(-64, 65, (T, E)) / 16.0).to(DT[dtype])


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (5, 31, 3), (7, 33, 32), (64, 64, 6), (9, 160, 6),
                                   (3, 256, 8), (2, 500, 4), (2, 1024, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_route_against_the_oracle(sigmoid, T, E, k, dtype):
    rng = np.random.default_rng(T + E)
    x = logits_of(rng, T, E, dtype)
    for renormalize, scale in ((True, 1.0), (False, 2.5)):
        ids, w = nv.route(x.to(DEV), k, score=nv.SCORE_SIGMOID if sigmoid else nv.SCORE_SOFTMAX,
                          renormalize=renormalize, weight_scale=scale)
        want_ids, want_w, _ = ol.route(x.double().numpy(), k, sigmoid, renormalize=renormalize, scale=scale)
        assert np.array_equal(host(ids), want_ids)
        # fp32: an exponential of 2 ulp, a sum of E terms, another of k, two divisions
        assert (np.abs(values(w) - want_w) <= (E + k + 8) * 2.0 ** -23 * np.abs(want_w) + 1e-30).all()


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 8, 4, 8), (96, 8, 3, 6), (256, 8, 4, 8), (32, 32, 5, 5),
                                                   (36, 2, 1, 8), (160, 16, 16, 4)])
def test_route_groups_and_bias(E, groups, top_groups, k, sigmoid):
    rng = np.random.default_rng(E + groups)
    T = 40
    x = logits_of(rng, T, E, "fp32")
    bias = (rng.permutation(E) / 64.0).astype(np.float32)
    args = dict(groups=groups, top_groups=top_groups)
    want_ids, want_w, rank = ol.route(x.double().numpy(), k, sigmoid, bias, **args)
    # keep the tokens whose ranks and group sums are further apart than fp32 rounding, or equal
    def clear(v):
        v = np.sort(v, axis=1)
        d = np.diff(np.where(np.isfinite(v), v, -1e3), axis=1)
        return ((d == 0) | (d > 1e-5)).all(axis=1)
    sc = ol.route(x.double().numpy(), k, sigmoid, bias)[2]
    two = np.sort(sc.reshape(T, groups, -1), axis=2)[:, :, ::-1][:, :, :2].sum(axis=2)
    fine = clear(rank) & clear(two)
    assert fine.sum() > T // 4
    ids, w = nv.route(x.to(DEV), k, score=nv.SCORE_SIGMOID if sigmoid else nv.SCORE_SOFTMAX, bias=gpu(bias), **args)
    assert np.array_equal(host(ids)[fine], want_ids[fine])
    assert (np.abs(values(w) - want_w)[fine] <= (E + k + 8) * 2.0 ** -23 * want_w[fine] + 1e-30).all()


def test_route_masks_and_extremes():
    E, k = 40, 4
    x = np.random.default_rng(1).standard_normal((9, E)).astype(np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 2:] = -np.inf                      # two left
    x[3] = np.finfo(np.float32).min         # the type's lowest value is a value: all equal
    x[4, 5] = np.inf
    x[5, 3], x[5, 9] = np.inf, np.inf
    x[6, :] = 0.0
    x[7, ::2] = -np.inf
    x[8] = 88 * np.sign(x[8])
    for sigmoid in (False, True):
        score = nv.SCORE_SIGMOID if sigmoid else nv.SCORE_SOFTMAX
        ids, w = nv.route(gpu(x), k, score=score)
        want_ids, want_w, _ = ol.route(x, k, sigmoid)
        assert np.array_equal(host(ids), want_ids)
        assert np.allclose(values(w), want_w, rtol=1e-5, atol=1e-30)
    bias = np.zeros(E, dtype=np.float32)
    bias[:20], bias[20] = -np.inf, np.nan
    ids, w = nv.route(gpu(x), k, score=nv.SCORE_SIGMOID, bias=gpu(bias), groups=4, top_groups=2)
    want_ids, want_w, _ = ol.route(x, k, True, bias, groups=4, top_groups=2)
    assert np.array_equal(host(ids), want_ids)
    assert np.allclose(values(w), want_w, rtol=1e-5, atol=1e-30)


def test_route_strided_rows_and_no_tokens():
    wide = logits_of(np.random.default_rng(2), 20, 100, "bf16").to(DEV)
    x = wide[:, 3:73]
    ids, w = nv.route(x, 5)
    a, b = nv.route(x.contiguous(), 5)
    assert torch.equal(ids, a) and torch.equal(w, b)
    ids, w = nv.route(wide[:0], 5)
    assert ids.shape == (0, 5) and w.shape == (0, 5)


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def choices(rng, T, k, E, holes=0.0):
    ids = np.argsort(rng.random((T, E)) - 0.5 * rng.random((1, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random(ids.shape) < holes] = -1
    return ids


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 64), (17, 3, 5), (200, 8, 16), (1000, 2, 1024), (700, 6, 9),
                                   (3000, 4, 37), (5000, 2, 2), (0, 4, 8)])
def test_moe_sort(T, k, E):
    rng = np.random.default_rng(T + E)
    ids = choices(rng, T, k, E, 0.05)
    if T > 3:
        ids[2], ids[3, 0] = -1, E  # a token without experts, an id out of range
    order = nv.moe_sort(gpu(ids), E)
    want, counts, starts = ol.moe_rows(ids, E, order["tile_rows"])
    assert np.array_equal(host(order["rows"]), want)
    assert np.array_equal(host(order["counts"]), counts)
    assert np.array_equal(host(order["starts"]), starts)
    assert want.max(initial=-1) < order["row_capacity"]


def test_moe_sort_all_to_one_expert():
    T, k, E = 900, 2, 64
    ids = np.full((T, k), 63, dtype=np.int32)
    order = nv.moe_sort(gpu(ids), E)
    want, _, _ = ol.moe_rows(ids, E, order["tile_rows"])
    assert np.array_equal(host(order["rows"]), want) and want.max() < order["row_capacity"]


@pytest.mark.parametrize("T,k,E,M,K", [(1, 2, 4, 128, 64), (5, 3, 8, 200, 288), (40, 2, 3, 136, 1056),
                                       (150, 4, 6, 256, 128), (600, 2, 3, 130, 96), (2000, 1, 2, 72, 64)])
def test_moe_gemm_exact_on_whole_numbers(T, k, E, M, K):
    rng = np.random.default_rng(T + M)
    ids = choices(rng, T, k, E, 0.1)
    order = nv.moe_sort(gpu(ids), E)
    x = rng.choice([0, 1, 2, 3, 4, 6], (T, K)) * rng.choice([-1.0, 1.0], (T, K))
    x[:, ::16] = 6
    q, sf = nv.quantize_rows(torch.from_numpy(x).to(DEV).bfloat16(), order)
    a, sfa = whole_matrix(rng, E, M, K)
    alpha = rng.choice([0.5, 1.0, 2.0], E).astype(np.float32)
    c = values(nv.moe_gemm(gpu(a), gpu(ol.atoms(sfa)), q, sf, order, alpha=gpu(alpha), dtype=torch.float32))
    w = ol.matrix(a, sfa)
    rows = host(order["rows"])
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e >= 0:
                assert np.array_equal(c[rows[t, j]], w[e] @ x[t] * alpha[e])


@pytest.mark.parametrize("act", [nv.ACT_SILU, nv.ACT_RELU, nv.ACT_GELU_TANH])
@pytest.mark.parametrize("T,k,E,F,K", [(1, 2, 4, 32, 64), (33, 3, 8, 96, 288), (150, 4, 6, 160, 128),
                                       (600, 2, 3, 64, 96)])
def test_moe_gated_gemm_codes(T, k, E, F, K, act):
    """gate and input are exact, so h is known to a few fp32 ulps: its codes are the oracle's
    wherever no boundary of the scale or of the code is that near."""
    rng = np.random.default_rng(T + F)
    ids = choices(rng, T, k, E, 0.1)
    order = nv.moe_sort(gpu(ids), E)
    x = rng.choice([0, 1, 2, 3, 4, 6], (T, K)) * rng.choice([-1.0, 1.0], (T, K))
    x[:, ::16] = 6
    xq, xs = nv.quantize_rows(torch.from_numpy(x).to(DEV).bfloat16(), order)
    a, sfa = whole_matrix(rng, E, 2 * F, K)
    alpha = np.full(E, 2.0 ** -6, dtype=np.float32)
    alpha[0] = 2.0 ** -8
    q, sf = nv.moe_gated_gemm(gpu(a), gpu(ol.atoms(sfa)), xq, xs, order, alpha=gpu(alpha), activation=act,
                              encode_scale=0.75)
    q, rows = host(q), host(order["rows"])
    pad = -(-F // 64) * 4
    sf = ol.from_atoms(host(sf), order["row_capacity"], pad)[0]
    w = ol.matrix(a, sfa)
    # 32 ulps of h; with relu h is a product of two whole numbers below 2^11 and 3/4: exact
    near = 0.0 if act == nv.ACT_RELU else 2.0 ** -19
    certain = []
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            u = w[e] @ x[t] * alpha[e]
            h = ol.activation(u[0::2], act) * u[1::2] * 0.75
            r = rows[t, j]
            assert not sf[r, F // 16:].any()
            lo, hi = (ol.quantize_values(h[None] * (1 + s * near)) for s in (-1, 1))
            same = lo[1][0] == hi[1][0]  # blocks whose scale is certain
            assert np.array_equal(sf[r, :F // 16][same], hi[1][0][same])
            cl, ch, got = (ol.e2m1_values(v).reshape(-1, 16) for v in (lo[0][0], hi[0][0], q[r]))
            sure = same[:, None] & (cl == ch)
            assert np.array_equal(got[sure], ch[sure])
            certain.append(sure.mean())
    assert np.mean(certain) > 0.9  # the comparison left little out


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,M", [(1, 1, 8), (5, 6, 264), (300, 8, 1024), (40, 32, 96)])
def test_moe_combine(T, k, M, wide, dtype):
    rng = np.random.default_rng(T + M)
    E = 64
    ids = choices(rng, T, k, E, 0.2)
    order = nv.moe_sort(gpu(ids), E)
    y = torch.randn(order["row_capacity"], M).to(torch.float32 if wide else DT[dtype])
    w = rng.random((T, k)).astype(np.float32)
    out = values(nv.moe_combine(y.to(DEV), order, gpu(w), dtype=DT[dtype]))
    rows = host(order["rows"])
    yv = y.double().numpy()
    terms = np.where(rows[..., None] >= 0, yv[rows] * w[..., None], 0.0)
    want = terms.sum(axis=1)
    tol = k * 2.0 ** -24 * np.abs(terms).sum(axis=1) + EPS[dtype] * np.abs(want) + TINY[dtype]
    assert (np.abs(out - want) <= tol * 1.01).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("T,k,E,D,F", [(1, 2, 4, 64, 32), (1, 6, 64, 2048, 256), (53, 8, 16, 288, 96),
                                       (300, 3, 5, 512, 160), (1500, 2, 7, 128, 64), (0, 2, 4, 64, 32)])
def test_moe_ffn_is_its_steps_and_near_the_formula(T, k, E, D, F, dtype):
    rng = np.random.default_rng(T + D)
    ids = choices(rng, T, k, E, 0.1 if T > 1 else 0.0)
    if T > 10:
        ids[3] = -1  # a token without experts: zeros
    w = rng.random((T, k)).astype(np.float32)
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(T)).to(DT[dtype])
    w1, s1 = any_matrix(rng, E, 2 * F, D)
    w2, s2 = any_matrix(rng, E, D, F)
    a1 = (0.02 / np.sqrt(D) * (1 + rng.random(E))).astype(np.float32)
    a2 = (0.02 / np.sqrt(F) * (1 + rng.random(E))).astype(np.float32)
    g = [gpu(v) for v in (w1, ol.atoms(s1), w2, ol.atoms(s2), a1, a2, ids, w)]
    out = nv.moe_ffn(x.to(DEV), g[6], g[7], *g[:4], alpha1=g[4], alpha2=g[5], encode_x=1.25, encode_h=8.0)
    if T == 0:
        assert out.shape == (0, D)
        return
    order = nv.moe_sort(g[6], E)
    xq, xs = nv.quantize_rows(x.to(DEV), order, 1.25)
    hq, hs = nv.moe_gated_gemm(g[0], g[1], xq, xs, order, alpha=g[4], encode_scale=8.0)
    # (an expert's output is fp32 up to 1024 choices)
    y = nv.moe_gemm(g[2], g[3], hq, hs, order, alpha=g[5], dtype=torch.float32 if T * k <= 1024 else DT[dtype])
    assert torch.equal(out, nv.moe_combine(y, order, g[7], dtype=DT[dtype]))
    # against the formula: with the kernel's own codes of h the second product is held to the
    # accuracy contract
    rows = host(order["rows"])
    cap, kb = order["row_capacity"], F // 16
    h = ol.matrix(host(hq), ol.from_atoms(host(hs), cap, kb)[0])
    m1, m2 = ol.matrix(w1, s1), ol.matrix(w2, s2)
    xv = ol.matrix(*ol.quantize(x.float().numpy(), 1.25))
    got = values(out)
    for t in range(0, T, max(1, T // 40)):
        want, tol = np.zeros(D), np.zeros(D)
        for j in range(k):
            e = ids[t, j]
            if e < 0:
                continue
            hv = h[rows[t, j]]
            yv = m2[e] @ hv * a2[e]
            want += w[t, j] * yv
            tol += w[t, j] * (1e-3 * np.abs(m2[e]) @ np.abs(hv) * a2[e] + EPS[dtype] * np.abs(yv) + TINY[dtype])
            # and h itself to one step of its codes: the largest is a third of the block's largest
            u = m1[e] @ xv[t] * a1[e]
            exact = ol.activation(u[0::2], 2) * u[1::2] * 8.0
            step = np.repeat(np.maximum(np.abs(exact), np.abs(hv)).reshape(-1, 16).max(axis=1), 16) / 3
            assert (np.abs(hv - exact) <= step + 2.0 ** -9).all()
        tol += EPS[dtype] * np.abs(want) * 1.01 + TINY[dtype]
        assert (np.abs(got[t] - want) <= tol).all()
    if T > 10:
        assert not got[3].any()


def test_moe_ffn_strided_rows_workspace_and_graph():
    rng = np.random.default_rng(11)
    T, k, E, D, F = 30, 2, 6, 128, 96
    wide = torch.randn(T, D + 24, device=DEV).bfloat16()
    x = wide[:, 8:8 + D]
    w1, s1 = any_matrix(rng, E, 2 * F, D)
    w2, s2 = any_matrix(rng, E, D, F)
    g = [gpu(v) for v in (w1, ol.atoms(s1), w2, ol.atoms(s2))]
    ids, w = gpu(choices(rng, T, k, E)), torch.rand(T, k, device=DEV)
    want = nv.moe_ffn(x.contiguous(), ids, w, *g, encode_h=2.0 ** -8)
    ws = torch.full((nv.nvfp4_moe_ffn_workspace_bytes(T, k, E, D, F),), 0xFF, dtype=torch.uint8, device=DEV)
    assert torch.equal(nv.moe_ffn(x, ids, w, *g, encode_h=2.0 ** -8, workspace=ws), want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.moe_ffn(x, ids, w, *g, encode_h=2.0 ** -8, workspace=ws)
    ids2 = gpu(choices(rng, T, k, E))
    want2 = nv.moe_ffn(x, ids2, w, *g, encode_h=2.0 ** -8)
    graph.replay()
    assert torch.equal(out, want)
    ids.copy_(ids2)
    graph.replay()
    assert torch.equal(out, want2)
