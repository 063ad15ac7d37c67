"""What the attention operators' torch calls hand to the library (CPU only: the launch is replaced)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import attention_ops as ao  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402


@pytest.fixture
def calls(monkeypatch):
    """The calls made: [(where, args)], structures as they are."""
    libbuild.build()
    made = []
    monkeypatch.setattr(ao, "_enqueue", lambda where, device, stream, *args: made.append((where, args)))
    return made


def options(args, kind):
    """The structure of that kind among a call's arguments."""
    for a in args:
        if hasattr(a, "_obj") and isinstance(a._obj, kind):
            return a._obj
    raise AssertionError("no such structure")


def problem(T=4, Hq=4, Hkv=2, D=64, B=2):
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16)
    cache = nv.kv_cache(2, Hkv, D, 16, device="cpu")
    return q, cache, torch.zeros(B, 2, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)


@pytest.mark.parametrize("window", [0, 1, 4096, (1 << 31) - 1])
def test_window_is_handed_over(calls, window):
    nv.attention(*problem(), window=window)
    assert options(calls[0][1], ao._AttentionOptions).window == window


@pytest.mark.parametrize("window", [1 << 31, (1 << 32) + 5, 1 << 40])
def test_windows_beyond_32_bits_see_every_token(calls, window):
    """No sequence has as many tokens: the widest window there is sees the same."""
    nv.attention(*problem(), window=window)
    assert options(calls[0][1], ao._AttentionOptions).window == (1 << 31) - 1
    calls.clear()
    lib = nv.library()
    seen = []

    class Fake:
        def nvfp4_attention(self, *args):
            seen.append(options(args, ao._AttentionOptions).window)
            return 0

    ao_library = ao.library
    ao.library = lambda: Fake()
    try:
        nv.nvfp4_attention(256, 1, 4, 4, 2, 64, 256, 2, 16, 256, 2, 256, 2, 256, 256, 1 << 20, window=window)
    finally:
        ao.library = ao_library
    assert seen == [(1 << 31) - 1] and lib is nv.library()


@pytest.mark.parametrize("kw", [dict(window=-1), dict(window=5 - (1 << 32)), dict(max_q=-1), dict(max_q=4 - (1 << 32))])
def test_negative_limits_are_refused(calls, kw):
    q, cache, table, lengths = problem()
    starts = torch.tensor([0, 2, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        nv.attention(q, cache, table, lengths, q_starts=starts, **kw)
    with pytest.raises(ValueError):
        nv.nvfp4_attention(256, 1, 4, 4, 2, 64, 256, 2, 16, 256, 2, 256, 2, 256, 256, 1 << 20, q_starts=256, **kw)
    assert not calls
