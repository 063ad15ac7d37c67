"""The torch calls on a stream given by name: what they allocate is neither still in use by the
current stream, nor handed out again while the call is to run."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402
from oracle import layer as ol  # noqa: E402
from test_gpu_layer import DEV, any_matrix, choices, gpu  # noqa: E402

pytestmark = pytest.mark.gpu
LATE = 40_000_000  # clocks of a kernel that only waits, ~20 ms: the calls are enqueued well before


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()
    # the fills below are to be enqueued at once
    torch.full((1 << 20,), 0xFF, dtype=torch.uint8, device=DEV).fill_(77)
    torch.cuda._sleep(1)


def calls():
    """{name: a function of stream}, each with outputs of some hundred KB and more, so that the
    allocator has blocks of their own for them."""
    rng = np.random.default_rng(1)
    T, k, E, D, F, M = 1200, 4, 8, 1024, 512, 1024
    x = torch.randn(T, D, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    ids, w = gpu(choices(rng, T, k, E)), torch.rand(T, k, device=DEV)
    w1, s1 = any_matrix(rng, E, 2 * F, D)
    w2, s2 = any_matrix(rng, E, D, F)
    m = [gpu(v) for v in (w1, ol.atoms(s1), w2, ol.atoms(s2))]
    a, sfa = any_matrix(rng, 1, M, D)
    a, sfa = gpu(a), gpu(ol.atoms(sfa))
    q, sf = nv.quantize(x)
    order = nv.moe_sort(ids, E)
    xq, xs = nv.quantize_rows(x, order)
    hq, hs = nv.moe_gated_gemm(m[0], m[1], xq, xs, order, encode_scale=2.0 ** -8)
    y = nv.moe_gemm(m[2], m[3], hq, hs, order, dtype=torch.bfloat16)
    logits = torch.randn(20000, 64, device=DEV)
    rows = torch.randint(0, 127, (4, 2000, 64), dtype=torch.uint8, device=DEV)
    held = order["rows"].flatten().long()
    kept = {"quantize_rows": lambda o: [o[0][held]], "moe_gemm": lambda o: [o[held]],
            "moe_gated_gemm": lambda o: [o[0][held]]}  # (other rows are not defined)
    # the GEMV: 64000 rows
    ga, gsa = any_matrix(rng, 8, 8000, 64)
    gb, gsb = any_matrix(rng, 8, 1, 64)
    gv = [gpu(v) for v in (ga, gb[:, 0], gsa, gsb[:, 0])]
    return {
        "quantize": lambda s: nv.quantize(x, stream=s),
        "dequantize": lambda s: nv.dequantize(q, sf, stream=s),
        "gemm": lambda s: nv.gemm(a, q.unsqueeze(0), sfa, sf, alpha=2.0 ** -8, stream=s),
        "route": lambda s: nv.route(logits, 8, stream=s),
        "moe_sort": lambda s: nv.moe_sort(ids, E, stream=s)["rows"],
        "quantize_rows": lambda s: nv.quantize_rows(x, order, stream=s),
        "moe_gated_gemm": lambda s: nv.moe_gated_gemm(m[0], m[1], xq, xs, order, encode_scale=2.0 ** -8, stream=s),
        "moe_gemm": lambda s: nv.moe_gemm(m[2], m[3], hq, hs, order, dtype=torch.bfloat16, stream=s),
        "moe_combine": lambda s: nv.moe_combine(y, order, w, stream=s),
        "moe_ffn": lambda s: nv.moe_ffn(x, ids, w, *m, encode_h=2.0 ** -8, stream=s),
        "gemv": lambda s: nv.gemv(*gv, stream=s),
        "repack_scales": lambda s: nv.repack_scales(rows, stream=s),
    }, kept


NAMES = ("quantize", "dequantize", "gemm", "route", "moe_sort", "quantize_rows", "moe_gated_gemm", "moe_gemm",
         "moe_combine", "moe_ffn", "gemv", "repack_scales")


@pytest.fixture(scope="module")
def ops():
    return calls()


def tensors(out):
    return list(out) if isinstance(out, tuple) else [out]


@pytest.mark.parametrize("form", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_not_memory_that_the_current_stream_still_writes(ops, name, form):
    call, kept = ops[0][name], ops[1].get(name, tensors)
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # blocks as large as the outputs, free again but to be written later on the current stream
    blocks = [torch.empty_like(t) for t in tensors(want)]
    torch.cuda._sleep(LATE)
    while blocks:
        blocks.pop(0).view(torch.uint8).fill_(77)
    got = call(side if form == "stream" else side.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(kept(got), kept(want)))


@pytest.mark.parametrize("name", ["moe_ffn", "gemm", "quantize"])
def test_what_a_call_drops_is_not_handed_out_before_it_has_run(ops, name):
    call = ops[0][name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(side):
        torch.cuda._sleep(LATE)
    got = call(side)
    # the current stream takes and writes blocks of all sizes meanwhile
    taken = [torch.full((1 << n,), 0xFF, dtype=torch.uint8, device=DEV) for n in range(12, 27) for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(tensors(got), tensors(want)))
    del taken


def test_results_used_and_dropped_on_the_current_stream_are_not_overwritten(ops):
    """The usual order: the current stream waits for the side's, uses the result and drops it; the
    next call on the side stream must not write over it before the use has run."""
    call = ops[0]["gemm"]
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(LATE)
    used = out.clone()
    del out
    with torch.cuda.stream(side):
        other = torch.zeros_like(want)
    torch.cuda.synchronize()
    assert torch.equal(used, want) and not other.any()


@pytest.mark.parametrize("offset", [0, 8, 1])
def test_every_call_sees_what_the_one_before_it_wrote(offset):
    """A chain of small calls that overwrite the same buffers, in a graph: each kernel may be launched
    before the one before it has ended, and reads only after that.  (Rows of 32-, 16- and 2-byte
    alignment take different loads.)  The values grow until the scales saturate, and stay there."""
    rng = np.random.default_rng(offset)
    N, K, steps = 40, 512, 60
    a, sfa = any_matrix(rng, 1, K, K)
    a, sfa = gpu(a), gpu(ol.atoms(sfa))
    wide = torch.zeros((N, K + 16), dtype=torch.bfloat16, device=DEV)
    x, c = wide[:, offset:offset + K], torch.empty((1, N, K), dtype=torch.bfloat16, device=DEV)
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=DEV)
    sf = torch.empty(nv.nvfp4_permuted_scale_bytes(N, K, 1), dtype=torch.uint8, device=DEV)
    back = torch.empty((N, K), dtype=torch.float32, device=DEV)
    stride = x.stride(0)
    start = torch.randn(N, K, device=DEV, generator=torch.Generator(device=DEV).manual_seed(offset)).bfloat16()

    def chain(wait):
        out = []

        def call(fn, *args, **kw):
            r = fn(*args, **kw)
            if wait:
                torch.cuda.synchronize()
            return r

        s = torch.cuda.current_stream().cuda_stream
        for _ in range(steps):
            call(nv.quantize, x, q=q, sf=sf)
            call(nv.dequantize, q, sf, x=back)
            call(nv.gemm, a, q.unsqueeze(0), sfa, sf, alpha=2.0 ** -6, c=c)
            # the rows of the next step, by the library's own kernels
            call(nv.quantize, c[0], encode_scale=0.5, q=q, sf=sf)
            call(nv.nvfp4_dequantize, q.data_ptr(), sf.data_ptr(), N, K, 1, x.data_ptr(), nv.DTYPE_BF16,
                 nv.SF_PERMUTED_128x4, 2.0, stride, s)
            i, v = call(nv.route, c[0, :, :64], 4)
            out += [back.clone(), c.clone(), i, v]
        return out

    x.copy_(start)
    want = chain(True)
    assert want[-3].isfinite().all() and want[-3].abs().max() > 0
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(5):
        x.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, t) for g, t in zip(got, want))
