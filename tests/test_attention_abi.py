"""The attention operators' refusals and host arithmetic (CPU only, no kernel launches)."""
import ctypes
import math

import numpy as np
import pytest

import nvfp4_block_scaled_gemv_gb300 as nv
from nvfp4_block_scaled_gemv_gb300 import attention_ops as ao
from nvfp4_block_scaled_gemv_gb300 import build as libbuild
from oracle import attention as oa

P = 256  # a pointer that no case below dereferences
V, U, A = nv.ERR_INVALID_VALUE, nv.ERR_UNSUPPORTED_SHAPE, nv.ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return nv.library()


@pytest.mark.parametrize("want,kw,opt", [
    (V, dict(dt=3), {}), (V, dict(T=-1), {}), (V, dict(H=-1), {}), (V, dict(D=-2), {}), (V, dict(pairs=-1), {}),
    (U, dict(pairs=0), {}), (V, dict(pairs=33), {}), (U, dict(pairs=513, D=2000), {}), (U, dict(D=65537), {}),
    (U, dict(H=65537), {}), (U, dict(H=65536, D=65536), {}), (U, dict(T=1 << 31), {}), (V, {}, dict(interleaved=2)), (V, {}, dict(inverse=-1)),
    (V, {}, dict(factor=math.inf)), (V, {}, dict(factor=math.nan)), (V, {}, dict(x_token_stride=-1)),
    (V, {}, dict(y_head_stride=(1 << 40) + 1)), (V, dict(x=None), {}), (V, dict(y=None), {}), (V, dict(pos=None), {}),
    (V, dict(table=None), {}), (A, dict(x=P + 1), {}), (A, dict(dt=2, y=P + 2), {}), (A, dict(pos=P + 2), {}),
    (A, dict(table=P + 4), {}), (V, {}, dict(x_token_stride=512, y_token_stride=1024)),
    (0, dict(T=0, x=None, y=None, pos=None), {}), (0, dict(H=0, x=None), {}),
])
def test_rope_refusals(lib, want, kw, opt):
    a = dict(x=P, dt=1, T=4, H=2, D=64, pos=P, table=P, pairs=32) | {n: v for n, v in kw.items() if n != "y"}
    o = ao._RopeOptions(**(dict(interleaved=0, inverse=0, factor=1.0, x_token_stride=0, x_head_stride=0,
                                y_token_stride=0, y_head_stride=0) | opt))
    assert lib.nvfp4_rope(*a.values(), ctypes.byref(o), kw.get("y", P), None) == want


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("want,kw,rows", [
    (V, dict(dt=3), {}), (V, dict(T=-1), {}), (V, dict(heads=0), {}), (V, dict(D=0), {}), (U, dict(D=96), {}),
    (U, dict(D=192), {}), (U, dict(D=512), {}), (V, dict(page=0), {}), (U, dict(page=24), {}), (U, dict(page=8), {}),
    (U, dict(page=(1 << 20) + 16), {}), (V, dict(pages=-1), {}), (U, dict(pages=1 << 31), {}),
    (U, dict(heads=65536), {}), (U, dict(pages=(1 << 31) - 1, heads=65535, page=1 << 20), {}),
    (U, dict(T=1 << 31), {}), (V, {}, dict(k_token_stride=-1)),
    (V, {}, dict(v_head_stride=-8)), (V, dict(slots=None), {}), (V, dict(cache=None), {}), (V, {}, dict(k=None, v=None)),
    (A, {}, dict(k=P + 1)), (A, {}, dict(v=P + 1)), (A, dict(slots=P + 4), {}), (A, dict(cache=P + 8), {}),
    (A, {}, dict(encode_k=P + 2)), (A, {}, dict(encode_v=P + 1)), (0, dict(T=0, slots=None, cache=None), dict(k=None)),
])
def test_cache_refusals(lib, want, kw, rows, write):
    a = dict(dt=1, T=4, heads=2, D=64, slots=P, cache=P, pages=3, page=16) | kw
    r = ao._KvRows(**(dict(k=P, v=P, encode_k=None, encode_v=None, k_token_stride=0, k_head_stride=0,
                           v_token_stride=0, v_head_stride=0) | rows))
    call = lib.nvfp4_kv_write if write else lib.nvfp4_kv_read
    assert call(ctypes.byref(r), *a.values(), None) == want


def test_cache_write_needs_both_sides(lib):
    for rows in (dict(k=None, v=P), dict(k=P, v=None)):
        r = ao._KvRows(encode_k=None, encode_v=None, **rows)
        assert lib.nvfp4_kv_write(ctypes.byref(r), 1, 4, 2, 64, P, P, 3, 16, None) == V
    assert lib.nvfp4_kv_write(None, 1, 4, 2, 64, P, P, 3, 16, None) == V


def test_cache_bytes(lib):
    size = nv.nvfp4_kv_cache_bytes
    assert size(3, 2, 128, 32) == oa.empty_cache(3, 2, 128, 32).nbytes
    assert size(1 << 20, 8, 128, 64) == (1 << 20) * 8 * 64 * 144 > 1 << 36
    assert size((1 << 31) - 1, 65535, 256, 1 << 20) == 0  # (more than 64 bits)
    assert size((1 << 26), 256, 256, 64) == (1 << 26) * 256 * 64 * 288
    assert size(0, 2, 64, 16) == 0 and size(3, 2, 96, 16) == 0 and size(3, 2, 64, 20) == 0 and size(-1, 2, 64, 16) == 0


@pytest.mark.parametrize("want,kw,opt", [
    (V, dict(dt=2), {}), (V, dict(dt=-1), {}), (V, dict(T=-1), {}), (V, dict(Hq=0), {}), (V, dict(Hkv=0), {}),
    (U, dict(Hq=5), {}), (U, dict(D=80), {}), (U, dict(page=40), {}), (V, dict(pages=-1), {}), (V, dict(mp=-1), {}),
    (U, dict(mp=1 << 27), {}), (U, dict(mp=(1 << 27) - 15), {}), (V, dict(mp=(1 << 27) - 16, q=None), {}),
    (U, dict(mp=1 << 26, B=64, T=64), {}), (U, dict(mp=1 << 23, B=32, T=32, Hq=128), {}), (V, dict(B=-1), {}), (V, dict(B=3), {}), (V, dict(B=0), {}),
    (U, dict(B=(1 << 20) + 1, T=(1 << 20) + 1), {}), (U, dict(T=1 << 30), {}), (V, {}, dict(max_q=3)),
    (V, {}, dict(max_q=-1)), (V, {}, dict(q_starts=P, max_q=5)), (V, {}, dict(scale=-1.0)),
    (V, {}, dict(scale=math.nan)), (V, {}, dict(scale=math.inf)), (V, {}, dict(causal=2)), (V, {}, dict(window=-1)),
    (V, {}, dict(window=4, causal=0)), (V, {}, dict(q_token_stride=-8)), (V, dict(q=None), {}), (V, dict(out=None), {}),
    (V, dict(lengths=None), {}), (V, dict(table=None), {}), (V, dict(cache=None), {}), (V, dict(ws=None), {}),
    (V, dict(size=0), {}), (A, dict(q=P + 8), {}), (A, {}, dict(q_token_stride=260)), (A, {}, dict(q_head_stride=68)),
    (A, dict(out=P + 8), {}), (A, dict(cache=P + 8), {}), (A, dict(ws=P + 128), {}), (A, dict(table=P + 2), {}),
    (A, dict(lengths=P + 2), {}), (A, {}, dict(q_starts=P + 2)), (A, {}, dict(encode_k=P + 2)),
    (A, {}, dict(encode_v=P + 2)), (A, {}, dict(lse=P + 2)), (0, dict(T=0, q=None, out=None, ws=None), {}),
    (0, dict(T=0, B=0, q=None), {}),
])
def test_attention_refusals(lib, want, kw, opt):
    a = dict(q=P, dt=1, T=4, Hq=4, Hkv=2, D=64, cache=P, pages=9, page=16, table=P, mp=7, lengths=P, B=2)
    a |= {n: v for n, v in kw.items() if n in a}
    o = ao._AttentionOptions(**(dict(scale=0.0, causal=1, window=0, max_q=0, q_starts=None, encode_k=None,
                                     encode_v=None, lse=None, q_token_stride=0, q_head_stride=0) | opt))
    size = kw.get("size", 1 << 30)
    assert lib.nvfp4_attention(*a.values(), ctypes.byref(o), kw.get("out", P), kw.get("ws", P), size, None) == want


def test_attention_workspace(lib):
    size = nv.nvfp4_attention_workspace_bytes
    one = size(1, 1, 8, 1, 128, 64, 100)
    assert 0 < one < 64 << 20
    # lengths and batch do not matter, the columns of a pass do
    assert size(64, 64, 64, 8, 128, 64, 10000) == one
    assert size(64, 16, 64, 8, 128, 64, 100) > one
    assert size(0, 4, 8, 1, 128, 64, 100) == 0 and size(3, 2, 8, 1, 128, 64, 100) == 0
    assert size(4, 2, 8, 3, 128, 64, 100) == 0


def test_rope_frequencies():
    f = nv.rope_frequencies(64)
    assert f[0] == 1.0 and np.allclose(np.diff(np.log(f)), -np.log(10000.0) / 32)
    assert np.allclose(nv.rope_frequencies(64, scaling="linear", factor=4.0), np.array(f) / 4)
    g = nv.rope_frequencies(64, scaling="base", factor=4.0)
    # the fastest pair stays, the slowest is divided by the factor
    assert g[0] == 1.0 and np.isclose(g[-1], f[-1] / 4)
    for kind in ("ramp", "bands"):
        g = np.array(nv.rope_frequencies(128, scaling=kind, factor=8.0, original=4096, low=1.0, high=32.0))
        f128 = np.array(nv.rope_frequencies(128))
        turns = 4096 * f128 / (2 * np.pi)
        # (the ramp starts and ends on whole pairs)
        assert np.allclose(g[turns > 40], f128[turns > 40]) and np.allclose(g[turns < 0.8], f128[turns < 0.8] / 8)
        assert (np.diff(g / f128) <= 1e-12).all() and (g <= f128 * (1 + 1e-12)).all() and (g >= f128 / 8 * (1 - 1e-12)).all()


@pytest.mark.parametrize("kw", [dict(rotary_dim=3), dict(rotary_dim=0), dict(scaling="half"), dict(base=1.0),
                                dict(factor=0.0), dict(scaling="ramp"), dict(scaling="bands", original=10, low=4.0, high=2.0),
                                dict(rotary_dim=2, scaling="base", factor=2.0), dict(base=math.inf)])
def test_rope_frequencies_refusals(kw):
    with pytest.raises(ValueError):
        nv.rope_frequencies(**(dict(rotary_dim=64) | kw))


def test_rope_table():
    torch = pytest.importorskip("torch")
    f = nv.rope_frequencies(96)
    table = nv.rope_table(96, device="cpu")
    assert table.dtype == torch.int64 and table.numel() == 48
    # the fraction of a turn at a far position, against whole-number arithmetic on the frequency
    from fractions import Fraction

    for i, t in enumerate(table.tolist()):
        exact = Fraction(f[i] / (2 * math.pi)) * 1000003
        got = Fraction((1000003 * t) % (1 << 64), 1 << 64)
        assert abs((exact - got + Fraction(1, 2)) % 1 - Fraction(1, 2)) < Fraction(1, 1 << 40)
    # any frequencies, negative and beyond a turn a position
    odd = nv.rope_table(frequencies=[-0.5, 7.0, 2 * math.pi - 0.5], device="cpu").tolist()
    assert all(-(1 << 63) <= t < 1 << 63 for t in odd)
    assert abs(odd[0] - odd[2]) < 1 << 16
    for bad in ([], [math.nan], [math.inf]):
        with pytest.raises(ValueError):
            nv.rope_table(frequencies=bad, device="cpu")


def test_torch_refusals_on_the_host():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64)
    table = nv.rope_table(64, device="cpu")
    pos = torch.zeros(4, dtype=torch.int32)
    for bad in (lambda: nv.rope(x[0], pos, table), lambda: nv.rope(x.transpose(1, 2), pos, table),
                lambda: nv.rope(x[..., :32], pos, table), lambda: nv.rope(x, pos[:3], table),
                lambda: nv.rope(x.expand(4, 2, 64)[:1].expand(4, 2, 64), pos, table),
                lambda: nv.rope(x, pos, table, out=x[:2]), lambda: nv.rope(x[:3], pos[:3], table, out=x[1:])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.rope(x.long(), pos, table), lambda: nv.rope(x, pos.long(), table),
                lambda: nv.rope(x, pos, table.int())):
        with pytest.raises(TypeError):
            bad()
    for kw in (dict(head_dim=96), dict(page_size=20), dict(heads=0), dict(pages=-1), dict(page_size=0)):
        with pytest.raises(ValueError):
            nv.kv_cache(**(dict(pages=2, heads=2, head_dim=64, page_size=16, device="cpu") | kw))
    cache = nv.kv_cache(2, 2, 64, 16, device="cpu")
    slots = torch.zeros(4, dtype=torch.int64)
    for bad in (lambda: nv.kv_write(x, x[:2], cache, slots), lambda: nv.kv_write(x[:, :1], x[:, :1], cache, slots),
                lambda: nv.kv_write(x, x, cache[0], slots), lambda: nv.kv_write(x, x, cache, slots[:3]),
                lambda: nv.kv_write(x, x, cache[..., :500], slots), lambda: nv.kv_read(cache, slots.view(2, 2)),
                lambda: nv.kv_write(x, x, cache, slots, encode_k=torch.ones(3))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        nv.kv_write(x, x, cache, slots.int())
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    t, n = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for bad in (lambda: nv.attention(q[:, :3], cache, t, n), lambda: nv.attention(q[:3], cache, t, n),
                lambda: nv.attention(q, cache, t[0], n), lambda: nv.attention(q, cache, t, n[:1]),
                lambda: nv.attention(q, cache, t, n, q_starts=n), lambda: nv.attention(q[..., :32], cache, t, n),
                lambda: nv.attention(q, cache, t, n, out=q[:2]), lambda: nv.attention(q, cache, t, n, out=q),
                lambda: nv.attention(q, cache, t, n, workspace=torch.zeros(16, dtype=torch.uint8)),
                # (a CPU tensor gets as far as the launch)
                lambda: nv.attention(q, cache, t, n)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: nv.attention(q.float(), cache, t, n), lambda: nv.attention(q, cache, t.long(), n)):
        with pytest.raises(TypeError):
            bad()


def test_oracle_attention_of_whole_numbers():
    """Equal scores give the mean, one far larger score its value, and the window its tokens."""
    k, v = np.zeros((6, 1, 64)), np.arange(6.0)[:, None, None] * np.ones((6, 1, 64))
    q = np.zeros((2, 2, 64))
    out, lse, _, _ = oa.attention(q, k, v, 1.0, 6)
    assert np.allclose(out[0], 2.0) and np.allclose(out[1], 2.5) and np.allclose(lse[1], np.log(6))
    out, _, _, _ = oa.attention(q, k, v, 1.0, 6, window=2)
    assert np.allclose(out[0], 3.5) and np.allclose(out[1], 4.5)
    out, lse, _, _ = oa.attention(q, k, v, 1.0, 1)  # the first query is before the sequence
    assert (out[0] == 0).all() and (lse[0] == -np.inf).all() and np.allclose(out[1], 0.0) and np.allclose(lse[1], 0)
    k[3] = 100.0
    q[:] = 1.0
    assert np.allclose(oa.attention(q, k, v, 1.0, 6)[0], 3.0)


def test_oracle_cache_places():
    """Every byte of a written cache is where the header says."""
    rng = np.random.default_rng(0)
    c = oa.empty_cache(3, 2, 128, 32, fill=0xAA)
    k, v = rng.standard_normal((2, 4, 2, 128)).astype(np.float32)
    oa.write(c, [5, 32 * 2 + 17, -1, 3 * 32], k, v)
    flat = c.reshape(-1)
    # token 17 of page 2, head 1, V, elements 64..79: byte 0 of the second plane's second row
    at = ((((2 * 2 + 1) * 2 + 1) * 2 + 1) * 2 + 1) * 576
    from oracle import layer as ol

    q, sf = ol.quantize(v[1, 1][None])
    assert flat[at + 32: at + 40].tolist() == q[0, 32:40].tolist() and flat[at + 512 + 4] == sf[0, 4]
    assert (c == 0xAA).mean() > 0.9  # (two tokens of 96)
    kv, vv = oa.values(c)
    assert np.array_equal(vv[2 * 32 + 17, 1], ol.matrix(q, sf)[0])
