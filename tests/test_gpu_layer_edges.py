"""The layer operators where a result can leave a type's range or be rounded once too often, on
the GPU, against formulas in 64 bits."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402
from oracle import layer as ol  # noqa: E402
from test_gpu_layer import DEV, DT, EPS, TINY, any_matrix, choices, gpu, host, whole_matrix  # noqa: E402

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



@pytest.mark.parametrize("T,k,E,tile", [(7, 3, 40, 16), (200, 2, 64, 16), (24, 2, 4, 32), (90, 2, 9, 64), (120, 2, 4, 128),
                                        (700, 2, 4, 256),
                                        (260, 4, 200, 16), (340, 8, 300, 32), (1100, 1, 40, 64)])
@pytest.mark.parametrize("uneven", [False, True])
def test_experts_rows_of_every_tile(T, k, E, tile, uneven):
    """The layer is its steps for every tile, one per expert or many (an expert that most choose)."""
    x, ids, w, m, a1 = experts(T, k, E, 128, 64, "bf16", T + k)
    if uneven:
        ids[:, 0] = E - 2
        ids[ids == 1] = -1
    assert nv.nvfp4_moe_shape(T, k, E)["tile_rows"] == tile
    order, y = outputs(x, ids, m, a1, a1, torch.float32)
    out = nv.moe_ffn(x, ids, w, *m, alpha1=a1, alpha2=a1, encode_h=8.0)
    assert torch.equal(out, nv.moe_combine(y, order, w, dtype=torch.bfloat16))



@pytest.mark.parametrize("T,k,E", [(70_000, 4, 100), (131_072, 8, 1024), (300_001, 1, 3)])
def test_sort_of_many_chunks_with_holes(T, k, E):
    """69 to 256 chunks of 4096 choices, some of them with no choice at all."""
    g = torch.Generator(device=DEV).manual_seed(T)
    ids = torch.randint(-1, E + 1, (T, k), dtype=torch.int32, device=DEV, generator=g)
    ids[T // 3:T // 3 + 20_000] = -1
    order = nv.moe_sort(ids, E)
    flat = ids.flatten().long()
    real = (flat >= 0) & (flat < E)
    tile, pitch = order["tile_rows"], max(order["tile_rows"], 128)
    counts = torch.bincount(flat[real], minlength=E)
    tiles = (counts + tile - 1) // tile
    first = tiles.cumsum(0) - tiles
    assert torch.equal(order["counts"].long(), counts) and torch.equal(order["starts"].long(), first * pitch)
    e, at = torch.where(real, flat, E).sort(stable=True)
    rank = torch.arange(T * k, device=DEV) - (counts.cumsum(0) - counts)[e.clamp(max=E - 1)]
    row = (first[e.clamp(max=E - 1)] + rank // tile) * pitch + rank % tile
    want = torch.empty_like(flat).scatter_(0, at, torch.where(e < E, row, -1))
    assert torch.equal(order["rows"].flatten().long(), want)


# ---------------------------------------------------------------------------
# the product's epilogue
# ---------------------------------------------------------------------------

U = 2.0 ** -24
PLAIN, RELU, SILU, GELU_TANH, GELU_ERF = range(5)
# finite values that overflow on the way (a cube, a product with log2 e) and their neighbours,
# the type's ends, and what is not finite
EXTREMES = [s * v for v in (1e4, 1e9, 1e12, 1.4e13, 1.6e13, 1e20, 1e30, 2.3e38, 2.5e38, 3.4028234e38, np.inf)
            for s in (1, -1)] + [np.nan, 0.0, -0.0, 87.0, -87.0, -87.5, -88.5, -89.0, -104.0]


def chosen(N, M, K, L, act):
    """(rows of b per tile, K split) of a call, by the library's own choice."""
    fn = nv.library()["_ZN5nvfp411choose_gemmEllllib"]  # choose_gemm(M, N, K, L, sms, activation)
    fn.argtypes, fn.restype = [ctypes.c_int64] * 4 + [ctypes.c_int, ctypes.c_bool], ctypes.c_uint64
    both = fn(M, N, K, L, torch.cuda.get_device_properties(0).multi_processor_count, act > RELU)
    return both & 0xFFFFFFFF, both >> 32


def formula(y, act):
    """(act(y) in 64 bits, a bound of the fp32 evaluation's error)."""
    y = y.double()
    if act == SILU or act == GELU_TANH:
        # a sigmoid of x: 16 units for the exponential, the sum and the quotient, |x| / 4 for log2 e,
        # 6 |x| for the roundings of x, where it is a polynomial of y; the quotient's end
        x = y if act == SILU else (8 / np.pi) ** 0.5 * (y + 0.044715 * y ** 3)
        want = y / (1 + torch.exp(-x))
        return want, (16 + (0.25 if act == SILU else 6.25) * x.abs().clamp(max=128)) * U * want.abs() + 2.0 ** -119
    if act == GELU_ERF:  # 1 + erf: absolute to an ulp or two of 1
        want = 0.5 * y * (1 + torch.erf(y / 2 ** 0.5))
        return want, 4 * U * (y.abs().clamp(max=1e30) + want.abs())
    if act == RELU:
        return torch.where(y > 0, y, torch.where(y.isnan(), y, 0.0)), 0 * y.nan_to_num(0, 0, 0)
    return y, 0 * y.nan_to_num(0, 0, 0)


def assert_epilogue(c, y, act, dtype):
    want, tol = formula(y, act)
    top = torch.finfo(DT[dtype]).max
    # values that round to an infinity of the type, and those that may do either
    over = want.abs() > top * (1 + EPS[dtype]) + tol
    edge = ~over & (want.abs() > top)
    got = c.double()
    assert torch.equal(got.isnan(), want.isnan())
    inf = float("inf")
    assert torch.equal(got[over], torch.where(want[over] > 0, inf, -inf))
    ok = (got - want).abs() <= tol + EPS[dtype] * want.abs() + TINY[dtype]
    ok |= over | want.isnan() | (edge & ((got.abs() == inf) | (got.abs() >= top)))
    assert ok.all(), (y[~ok][:4], c[~ok][:4], want[~ok][:4])


def exact_case(N, M, K, L, alpha=2.0 ** -6, bias=None):
    """(a, b and their scales, bias, alpha * sums + bias in fp32) of whole-number matrices, alpha a power
    of two and the bias, if it is not given, in 64ths: exact but for a given bias's sum."""
    rng = np.random.default_rng(N + M + K)
    a, sfa = whole_matrix(rng, L, M, K)
    b, sfb = whole_matrix(rng, L, N, K)
    if bias is None:
        bias = gpu(rng.integers(-512, 513, (L, M)).astype(np.float32) / 64)
    at, bt = (torch.from_numpy(ol.matrix(*m)).float().to(DEV) for m in ((a, sfa), (b, sfb)))
    # (whole numbers below 2^24: fp32 products are exact in any order)
    y = (torch.bmm(bt, at.transpose(1, 2)) * alpha).double() + bias.double().unsqueeze(1)
    return [gpu(a), gpu(b), gpu(ol.atoms(sfa)), gpu(ol.atoms(sfb))], bias, y.float()


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("act", range(5))
def test_activations_of_extreme_values(act, dtype):
    """Through the bias: the one-SM kernel, the pair kernel and the product without K."""
    for N, M, K, L, tile in ((40, 140, 64, 2, 64), (257, 4096, 4096, 2, 256)):
        assert chosen(N, M, K, L, act)[0] == tile
        bias = torch.tensor(EXTREMES, dtype=torch.float32, device=DEV).repeat(-(-L * M // len(EXTREMES)))
        bias = bias[:L * M].view(L, M)
        t, bias, y = exact_case(N, M, K, L, 2.0 ** -10, bias)
        assert_epilogue(nv.gemm(*t, alpha=2.0 ** -10, bias=bias, activation=act, dtype=DT[dtype]), y, act, dtype)
    e = torch.empty(0, dtype=torch.uint8, device=DEV)
    y = torch.tensor(EXTREMES, dtype=torch.float32, device=DEV).view(1, -1)
    c = nv.gemm(e.view(1, y.numel(), 0), e.view(1, 1, 0), e, e, bias=y, activation=act, dtype=DT[dtype])[0]
    want = formula(y, act)[0].to(DT[dtype])
    big = y.abs() >= 1e4
    assert torch.equal(c[big].nan_to_num(-7), want[big].nan_to_num(-7))


@pytest.mark.parametrize("act", [nv.ACT_SILU, nv.ACT_GELU_TANH])
@pytest.mark.parametrize("T,k,E,F,K", [(33, 3, 8, 96, 288), (600, 2, 3, 64, 96)])
def test_gated_product_of_large_gates(T, k, E, F, K, act):
    """Gates of 2^36 times whole numbers: the sigmoid is 0 or 1, and the scaled h is within the
    scales' range."""
    rng = np.random.default_rng(T)
    ids = choices(rng, T, k, E)
    order = nv.moe_sort(gpu(ids), E)
    x = rng.choice([0, 1, 2, 3, 4, 6], (T, K)) * rng.choice([-1.0, 1.0], (T, K))
    x[:, ::16] = 6
    xq, xs = nv.quantize_rows(torch.from_numpy(x).to(DEV).bfloat16(), order)
    a, sfa = whole_matrix(rng, E, 2 * F, K)
    alpha, encode = 2.0 ** 36, 2.0 ** -88
    q, sf = nv.moe_gated_gemm(gpu(a), gpu(ol.atoms(sfa)), xq, xs, order, alpha=torch.full((E,), alpha, device=DEV),
                              activation=act, encode_scale=encode)
    rows, w = host(order["rows"]), ol.matrix(a, sfa)
    sf = ol.from_atoms(host(sf), order["row_capacity"], -(-F // 64) * 4)[0][:, :F // 16]
    q = host(q)
    for t in range(T):
        for j in range(k):
            u = w[ids[t, j]] @ x[t]
            # a gate that is 0 gives 0; a quotient by 1 is exact to two ulps
            h = np.maximum(u[0::2], 0) * u[1::2] * (alpha * alpha * encode)
            lo, hi = (ol.quantize_values(h[None] * (1 + s * 2.0 ** -21)) for s in (-1, 1))
            same = lo[1][0] == hi[1][0]
            assert (sf[rows[t, j]] != 0x7F).all() and np.array_equal(sf[rows[t, j]][same], hi[1][0][same])
            cl, ch, got = (ol.e2m1_values(v).reshape(-1, 16) for v in (lo[0][0], hi[0][0], q[rows[t, j]]))
            sure = same[:, None] & (cl == ch)
            assert np.array_equal(got[sure], ch[sure]) and sure.mean() > 0.5


# (N, M, K, L): rows per tile and K split, without an activation and with one that has an exponential
PATHS = {(1, 513, 2080, 1): ((16, 2), (16, 4)), (16, 4096, 4096, 1): ((16, 4),) * 2,
         (30, 2048, 4128, 2): ((32, 4),) * 2, (40, 1000, 8192, 1): ((64, 2),) * 2,
         (100, 1000, 8192, 1): ((128, 2),) * 2, (9, 20000, 544, 1): ((16, 1),) * 2,
         (20, 20000, 544, 1): ((32, 1),) * 2, (40, 20000, 544, 1): ((64, 1),) * 2,
         (100, 7000, 2048, 1): ((128, 1),) * 2,
         # pairs of SMs: rows of c that TMA can store, and rows that it cannot
         (257, 4096, 4096, 2): ((256, 1),) * 2, (257, 4101, 4096, 2): ((256, 1),) * 2,
         (1153, 4224, 4096, 2): ((256, 1),) * 2}


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "x".join(map(str, p)))
def test_epilogue_of_every_kernel(path):
    """Scaling, bias, each activation and each type where K is split, where it is not, and on pairs."""
    t, bias, y = exact_case(*path)
    for act in range(5):
        assert chosen(*path, act) == PATHS[path][act > RELU]
        for dtype in DT:
            c = nv.gemm(*t, alpha=2.0 ** -6, bias=bias, activation=act, dtype=DT[dtype])
            assert_epilogue(c, y, act, dtype)


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("gap", [8, 2, 1])
@pytest.mark.parametrize("path", [(257, 4096, 4096, 2), (16, 4096, 4096, 1), (100, 7000, 2048, 1)],
                         ids=lambda p: "x".join(map(str, p)))
def test_epilogue_into_rows_with_gaps(path, gap, dtype):
    """Rows of c that start on 16 bytes (TMA stores them on pairs), on two elements, on one."""
    N, M, K, L = path
    t, bias, y = exact_case(*path)
    out = torch.full((L, N, M + gap), -77.0, dtype=DT[dtype], device=DEV)
    nv.nvfp4_gemm(*[x.data_ptr() for x in t], out.data_ptr(), M, N, K, L, alpha=2.0 ** -6, bias=bias.data_ptr(),
                  activation=GELU_TANH, c_dtype={"fp16": nv.DTYPE_FP16, "bf16": nv.DTYPE_BF16, "fp32": nv.DTYPE_FP32}[dtype],
                  c_row_stride=M + gap, stream=torch.cuda.current_stream().cuda_stream)
    assert_epilogue(out[..., :M], y, GELU_TANH, dtype)
    assert (out[..., M:] == -77).all()


@pytest.mark.parametrize("N", [1, 2, 16])
def test_gemm_of_folded_scales_is_the_small_product_of_signed_ones(N):
    """The two products for up to 16 rows: one takes signed scales, the other magnitudes."""
    M, K, L = 300, 512, 2
    rng = np.random.default_rng(N)
    a, sfa = whole_matrix(rng, L, M, K)
    b, sfb = whole_matrix(rng, L, N, K)
    sfa, sfb = (s | (rng.integers(0, 2, s.shape) << 7).astype(np.uint8) for s in (sfa, sfb))
    t = [gpu(a), gpu(b), gpu(ol.atoms(sfa)), gpu(ol.atoms(sfb))]
    small = torch.empty((L, N, M), dtype=torch.float16, device=DEV)
    nv.nvfp4_gemm_small_n(*[x.data_ptr() for x in t], small.data_ptr(), M, N, K, L, alpha=2.0 ** -2,
                          stream=torch.cuda.current_stream().cuda_stream)
    assert not torch.equal(nv.gemm(*t, alpha=2.0 ** -2), small)  # (the signs are ignored)
    for m, s in ((0, 2), (1, 3)):
        nv.fold_scale_signs(t[m], t[s])
    # whole numbers below 2^24, a power of two, one rounding
    assert torch.equal(nv.gemm(*t, alpha=2.0 ** -2), small)
