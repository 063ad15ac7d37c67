"""The layer operators' refusals and host arithmetic (CPU only, no kernel launches)."""
import ctypes

import pytest

import nvfp4_block_scaled_gemv_gb300 as nv
from nvfp4_block_scaled_gemv_gb300 import build as libbuild
from nvfp4_block_scaled_gemv_gb300 import layer

P = 256  # a pointer that no case below dereferences
V, U, A = nv.ERR_INVALID_VALUE, nv.ERR_UNSUPPORTED_SHAPE, nv.ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return nv.library()


def quantize(lib, x=P, dt=1, stride=0, rows=4, K=64, L=1, enc=1.0, q=P, sf=P, layout=1, rmap=None, copies=0,
             q_rows=0):
    return lib.nvfp4_quantize(x, dt, stride, rows, K, L, enc, q, sf, layout, rmap, copies, q_rows, None)


@pytest.mark.parametrize("want,kw", [
    (V, dict(dt=3)), (V, dict(dt=-1)), (V, dict(rows=-1)), (V, dict(K=-16)), (V, dict(L=-1)),
    (V, dict(stride=63)), (V, dict(stride=-1)), (V, dict(layout=2)), (V, dict(enc=0.0)), (V, dict(enc=-1.0)),
    (V, dict(enc=float("nan"))), (V, dict(enc=float("inf"))), (V, dict(x=None)), (V, dict(q=None)),
    (V, dict(sf=None)), (V, dict(rmap=P)), (V, dict(rmap=P, copies=1, q_rows=-1)),
    (V, dict(rmap=P, copies=1, q_rows=4, L=2)), (U, dict(rmap=P, copies=33, q_rows=4)),
    (U, dict(K=24)), (U, dict(K=(1 << 30) + 16)), (U, dict(rows=1 << 31)), (U, dict(rows=1 << 30, L=1 << 11)),
    (A, dict(x=P + 1)), (A, dict(dt=2, x=P + 2)), (A, dict(q=P + 4)), (A, dict(sf=P + 2)),
    (A, dict(rmap=P + 2, copies=1, q_rows=4)),
    (0, dict(rows=0, x=None, q=None, sf=None)), (0, dict(K=0, x=None)), (0, dict(L=0, sf=None)),
])
def test_quantize_refusals(lib, want, kw):
    assert quantize(lib, **kw) == want


@pytest.mark.parametrize("want,kw", [
    (V, dict(dt=5)), (V, dict(layout=-1)), (V, dict(rows=-1)), (V, dict(x=None)), (V, dict(stride=3)),
    (U, dict(K=8)), (A, dict(x=P + 1)), (A, dict(q=P + 1)), (0, dict(rows=0, x=None)),
])
def test_dequantize_refusals(lib, want, kw):
    a = dict(q=P, sf=P, layout=1, rows=4, K=64, L=1, scale=1.0, x=P, dt=1, stride=0) | kw
    assert lib.nvfp4_dequantize(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (V, dict(a=None)), (V, dict(sf=None)), (V, dict(layout=7)), (V, dict(L=-1)), (U, dict(K=20)),
    (A, dict(a=P + 4)), (0, dict(K=0, a=None, sf=None)),
])
def test_fold_scale_signs_refusals(lib, want, kw):
    a = dict(a=P, sf=P, layout=1, rows=4, K=64, L=1) | kw
    assert lib.nvfp4_fold_scale_signs(*a.values(), None) == want


@pytest.mark.parametrize("want,kw,opt", [
    (V, dict(M=-1), {}), (V, dict(N=-1), {}), (V, dict(K=-32), {}), (V, dict(L=-1), {}),
    (U, dict(K=48), {}), (U, dict(K=(1 << 30) + 32), {}), (U, dict(M=1 << 31), {}), (U, dict(N=1 << 31), {}),
    (U, dict(M=1 << 30, L=1 << 11), {}), (U, dict(M=1 << 22, K=1 << 20), {}),
    (U, dict(M=1 << 22, N=1 << 21, L=1), {}),
    (V, {}, dict(activation=5)), (V, {}, dict(activation=-1)), (V, {}, dict(c_dtype=3)),
    (V, {}, dict(c_row_stride=7)), (V, dict(c=None), {}), (V, dict(a=None), {}), (V, dict(sfb=None), {}),
    (A, dict(a=P + 8), {}), (A, dict(b=P + 8), {}), (A, dict(sfa=P + 8), {}), (A, dict(sfb=P + 8), {}),
    (A, dict(c=P + 1), {}), (A, dict(c=P + 2), dict(c_dtype=2)), (A, {}, dict(bias=P + 2)),
    (0, dict(M=0, a=None, c=None), {}), (0, dict(N=0, b=None, c=None), {}), (0, dict(L=0, c=None), {}),
])
def test_gemm_refusals(lib, want, kw, opt):
    a = dict(a=P, b=P, sfa=P, sfb=P, c=P, M=8, N=4, K=64, L=1) | kw
    o = layer._GemmOptions(**(dict(alpha=1.0, bias=None, activation=0, c_dtype=0, c_row_stride=0) | opt))
    assert lib.nvfp4_gemm(*a.values(), ctypes.byref(o), None) == want


def test_gemm_plan(lib):
    plan = nv.nvfp4_gemm_plan
    # one tile of b's rows as long as it holds them, split while SMs are idle
    assert plan(4096, 1, 4096) == {"tile_rows": 16, "k_split": 4}
    assert plan(4096, 17, 4096)["tile_rows"] == 32 and plan(4096, 64, 4096)["tile_rows"] == 64
    assert plan(65536, 16, 4096) == {"tile_rows": 16, "k_split": 1}
    for M, N, K in ((4096, 1, 256), (100, 7, 32), (128, 100, 500 * 32)):
        p = plan(M, N, K)
        stages = -(-K // 256)
        assert p["k_split"] == 1 or stages >= 2 * p["k_split"]
        assert -(-M // 128) * -(-N // p["tile_rows"]) * p["k_split"] <= 152
    # tiles below 128 rows start on no scale atom but the first
    for N in (129, 200, 333, 1000, 8192):
        assert plan(4096, N, 2048)["tile_rows"] in (128, 256)
    assert plan(8192, 8192, 8192) == {"tile_rows": 256, "k_split": 1}
    r = ctypes.byref(ctypes.c_int())
    assert lib.nvfp4_gemm_plan(8, 8, 64, 1, 152, None, r) == V
    assert lib.nvfp4_gemm_plan(8, 8, 64, 1, 1, r, r) == V
    assert lib.nvfp4_gemm_plan(8, 8, 40, 1, 152, r, r) == U


@pytest.mark.parametrize("N,M,K,L,rows,split", [
    (320, 20000, 8192, 1, 256, 1), (560, 12000, 8224, 1, 256, 1),  # narrow last tiles of pairs
    (320, 4096, 1024, 3, 128, 1), (310, 9000, 1024, 1, 128, 1),    # too little K for a pair's epilogue
    (40, 3000, 4128, 1, 64, 2), (128, 9000, 4128, 1, 128, 1), (500, 1000, 4128, 1, 128, 1)])
def test_gemm_plan_takes_the_faster_tile(lib, N, M, K, L, rows, split):
    """Shapes on which another tile or split measured 2 to 60% slower."""
    assert nv.nvfp4_gemm_plan(M, N, K, L) == {"tile_rows": rows, "k_split": split}


@pytest.mark.parametrize("want,kw,opt", [
    (V, dict(dt=3), {}), (V, dict(T=-1), {}), (V, dict(E=0), {}), (V, dict(k=0), {}), (V, dict(stride=31), {}),
    (U, dict(E=1025, k=4), {}), (U, dict(k=33, E=64), {}), (U, dict(k=33), {}), (U, {}, dict(groups=5)),
    (U, dict(E=66), dict(groups=33)), (V, {}, dict(groups=0)), (V, {}, dict(groups=4, top_groups=5)),
    (V, {}, dict(top_groups=0)), (V, {}, dict(score=2)), (V, dict(x=None), {}), (V, dict(ids=None), {}),
    (V, dict(w=None), {}), (A, dict(x=P + 2), {}), (A, dict(ids=P + 2), {}), (A, dict(w=P + 1), {}),
    (A, {}, dict(bias=P + 1)), (0, dict(T=0, x=None, ids=None, w=None), {}),
])
def test_route_refusals(lib, want, kw, opt):
    a = dict(x=P, dt=2, stride=0, T=4, E=32, k=4) | {n: v for n, v in kw.items() if n not in ("ids", "w")}
    o = layer._RouteOptions(**(dict(score=0, bias=None, groups=1, top_groups=1, renormalize=1,
                                    weight_scale=1.0) | opt))
    assert lib.nvfp4_route(*a.values(), ctypes.byref(o), kw.get("ids", P), kw.get("w", P), None) == want


@pytest.mark.parametrize("want,T,k,E", [(V, -1, 1, 4), (V, 4, 0, 4), (V, 4, 1, 0), (U, 4, 5, 4), (U, 4, 33, 64),
                                        (U, 4, 1, 1025), (U, (1 << 24) + 1, 1, 4), (0, 0, 1, 4), (0, 1, 32, 1024)])
def test_moe_shape_refusals(lib, want, T, k, E):
    assert lib.nvfp4_moe_shape(T, k, E, ctypes.byref(layer._MoeShape())) == want
    assert lib.nvfp4_moe_shape(1, 1, 1, None) == V
    if want:
        assert nv.nvfp4_moe_ffn_workspace_bytes(T, k, E, 64, 64) == 0


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (7, 2, 3), (100, 8, 64), (4096, 8, 64), (9999, 4, 100),
                                   (300000, 8, 1024)])
def test_moe_shape_holds_any_choice(T, k, E):
    """The capacity covers the worst split of the choices: as many experts as can be with one
    row more than whole tiles."""
    s = nv.nvfp4_moe_shape(T, k, E)
    tile, n = s["tile_rows"], T * k
    assert tile in (16, 32, 64, 128, 256)
    pitch = max(tile, 128)
    assert s["row_capacity"] % 128 == 0
    # E' experts with a last tile of one row each, the others' choices in whole tiles
    for split in {1, min(E, n), min(E, max(1, n // tile))}:
        tiles = split + max(0, n - split) // tile
        assert tiles * pitch <= s["row_capacity"]
    assert s["plan_bytes"] >= 16 * (s["row_capacity"] // pitch) + 16


@pytest.mark.parametrize("want,kw", [
    (V, dict(ids=None)), (V, dict(rows=None)), (V, dict(counts=None)), (V, dict(starts=None)),
    (V, dict(plan=None)), (A, dict(ids=P + 2)), (A, dict(rows=P + 1)), (A, dict(plan=P + 8)), (V, dict(T=-1)),
    (U, dict(k=9)),
])
def test_moe_sort_refusals(lib, want, kw):
    a = dict(ids=P, T=4, k=2, E=8, rows=P, counts=P, starts=P, plan=P) | kw
    assert lib.nvfp4_moe_sort(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (V, dict(a=None)), (V, dict(sfa=None)), (V, dict(b=None)), (V, dict(sfb=None)), (V, dict(plan=None)),
    (V, dict(c=None)), (V, dict(M=-1)), (V, dict(act=9)), (V, dict(dt=4)), (U, dict(K=0)), (U, dict(K=40)),
    (A, dict(a=P + 8)), (A, dict(plan=P + 4)), (A, dict(c=P + 1)), (A, dict(alpha=P + 2)),
    (U, dict(T=1 << 23, M=1 << 23)), (0, dict(M=0, c=None)), (0, dict(T=0, plan=None)),
])
def test_moe_gemm_refusals(lib, want, kw):
    a = dict(a=P, sfa=P, b=P, sfb=P, plan=P, T=4, k=2, E=8, M=128, K=64, alpha=None, act=0, c=P, dt=0) | kw
    assert lib.nvfp4_moe_gemm(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (V, dict(q=None)), (V, dict(sf=None)), (V, dict(F=-32)), (V, dict(act=-1)), (V, dict(enc=0.0)),
    (U, dict(F=48)), (U, dict(K=0)), (A, dict(q=P + 8)), (A, dict(sf=P + 8)), (0, dict(F=0, q=None)),
])
def test_moe_gated_gemm_refusals(lib, want, kw):
    a = dict(a=P, sfa=P, b=P, sfb=P, plan=P, T=4, k=2, E=8, F=64, K=64, alpha=None, act=2, enc=1.0, q=P,
             sf=P) | kw
    assert lib.nvfp4_moe_gated_gemm(*a.values(), None) == want


@pytest.mark.parametrize("want,kw", [
    (V, dict(y=None)), (V, dict(rows=None)), (V, dict(w=None)), (V, dict(out=None)), (V, dict(dt=2)),
    (V, dict(ydt=1)), (V, dict(ydt=3)), (V, dict(T=-1)), (U, dict(M=12)), (U, dict(k=33)), (A, dict(y=P + 8)), (A, dict(out=P + 8)),
    (0, dict(T=0, y=None)), (0, dict(M=0, out=None)),
])
def test_moe_combine_refusals(lib, want, kw):
    a = dict(y=P, ydt=0, rows=P, w=P, T=4, k=2, M=64, out=P, dt=0) | kw
    assert lib.nvfp4_moe_combine(*a.values(), None) == want


@pytest.mark.parametrize("want,kw,opt", [
    (V, dict(x=None), {}), (V, dict(ids=None), {}), (V, dict(w=None), {}), (V, dict(w1=None), {}),
    (V, dict(sf2=None), {}), (V, dict(out=None), {}), (V, dict(ws=None), {}), (V, dict(bytes=1000), {}),
    (V, dict(dt=2), {}), (V, dict(stride=63), {}), (U, dict(D=48), {}), (U, dict(F=16), {}), (U, dict(D=0), {}),
    (U, dict(k=9), {}), (V, {}, dict(activation=5)), (V, {}, dict(encode_x=0.0)),
    (V, {}, dict(encode_h=float("nan"))), (A, dict(x=P + 1), {}), (A, dict(out=P + 2), {}), (A, dict(w1=P + 4), {}),
    (A, dict(ws=P + 16), {}), (A, {}, dict(alpha1=P + 2)), (0, dict(T=0, x=None, out=None, ws=None), {}),
])
def test_moe_ffn_refusals(lib, want, kw, opt):
    a = dict(x=P, dt=1, stride=0, ids=P, w=P, w1=P, sf1=P, w2=P, sf2=P, T=4, k=2, E=8, D=64, F=64) | {
        n: v for n, v in kw.items() if n not in ("out", "ws", "bytes")}
    o = layer._MoeOptions(**(dict(alpha1=None, alpha2=None, encode_x=1.0, encode_h=1.0, activation=2) | opt))
    rest = (kw.get("out", P), kw.get("ws", P), kw.get("bytes", 1 << 40))
    assert lib.nvfp4_moe_ffn(*a.values(), ctypes.byref(o), *rest, None) == want


def test_torch_calls_check_their_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 64))
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    with pytest.raises(TypeError):
        nv.quantize(x.double())
    with pytest.raises(ValueError):
        nv.quantize(torch.zeros((4, 24)))
    with pytest.raises(ValueError):
        nv.quantize(x.t())
    with pytest.raises(ValueError):
        nv.quantize(x[:1].expand(4, 64))
    with pytest.raises(ValueError):
        nv.dequantize(u8, torch.zeros(3, dtype=torch.uint8))
    with pytest.raises(ValueError):
        nv.gemm(u8, u8, u8, u8)
    with pytest.raises(TypeError):
        nv.gemm(u8[None], u8[None], x, x)
    with pytest.raises(TypeError):
        nv.route(torch.zeros((4, 8), dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="CUDA device"):
        nv.route(torch.zeros((4, 8)), 2)
    with pytest.raises(ValueError, match="CUDA device"):
        nv.quantize(x)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_route(P, nv.DTYPE_FP32, 4, 8, 9, P, P)
    with pytest.raises(TypeError):
        nv.moe_sort(torch.zeros((4, 2), dtype=torch.int64), 8)
    with pytest.raises(TypeError):
        nv.moe_ffn(x, None, None, None, None, None, None)
