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


def one_of(buffer, T, H, D, at=0):
    """A view [T, H, D] whose rows lie at odd distances."""
    return buffer[:T, at: at + H * D].unflatten(1, (H, D))


def test_strides_that_nothing_steps_by(calls):
    """A single token's distance to the next, and a single head's, may be any: the call is not refused for it, and does
    not take a slower path."""
    _, cache, table, lengths = problem(B=1)
    row = torch.zeros(1, 4 * 64 + 3, dtype=torch.bfloat16)
    out = nv.attention(one_of(row, 1, 4, 64), cache, table, lengths)
    opt = options(calls[0][1], ao._AttentionOptions)
    assert out.shape == (1, 4, 64) and opt.q_token_stride % 8 == 0 and opt.q_head_stride == 64
    cache = nv.kv_cache(2, 1, 64, 16, device="cpu")
    flat = torch.zeros(3 * 72 + 8, dtype=torch.bfloat16)
    for head in (65, 1, 67):
        q = flat.as_strided((3, 1, 64), (72, head, 1))
        calls.clear()
        nv.attention(q, cache, torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
        opt = options(calls[0][1], ao._AttentionOptions)
        assert opt.q_token_stride == 72 and opt.q_head_stride % 8 == 0
        calls.clear()
        nv.kv_write(q, q, cache, torch.zeros(3, dtype=torch.int64))
        rows = options(calls[0][1], ao._KvRows)
        assert rows.k_token_stride == rows.v_token_stride == 72 and rows.k_head_stride % 8 == rows.v_head_stride % 8 == 0
        calls.clear()
        table64 = nv.rope_table(64, device="cpu")
        nv.rope(q, torch.zeros(3, dtype=torch.int32), table64)
        opt = options(calls[0][1], ao._RopeOptions)
        assert opt.x_token_stride == 72 and opt.x_head_stride % 8 == 0
    # a stride that is stepped by is still looked at
    wide = torch.zeros(2, 4 * 64 + 3, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="aligned"):
        nv.attention(one_of(wide, 2, 4, 64), nv.kv_cache(2, 2, 64, 16, device="cpu"), torch.zeros(2, 2, dtype=torch.int32),
                     torch.zeros(2, dtype=torch.int32))


def test_strides_of_rows_in_place(calls):
    """A single token turned in place: both sides have the same strides."""
    row = torch.zeros(1, 3 * 64 + 5)
    x = one_of(row, 1, 3, 64)
    assert nv.rope(x, torch.zeros(1, dtype=torch.int32), nv.rope_table(64, device="cpu"), out=x) is x
    opt = options(calls[0][1], ao._RopeOptions)
    assert (opt.x_token_stride, opt.x_head_stride) == (opt.y_token_stride, opt.y_head_stride)


@pytest.mark.parametrize("scale,given", [(0.0, 0.0), (0.125, 0.125), (2.0 ** -140, 2.0 ** -140), (1e-60, 2.0 ** -149)])
def test_scale_is_not_taken_for_the_default(calls, scale, given):
    """0 means 1 / sqrt(D); a scale too small for fp32 is the smallest there is, with which no scores differ either."""
    nv.attention(*problem(), scale=scale)
    assert options(calls[0][1], ao._AttentionOptions).scale == given
