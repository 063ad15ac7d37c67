"""What the layer calls promise about sizes, options and footprints (CPU only, no launches)."""
import ctypes

import pytest

import nvfp4_block_scaled_gemv_gb300 as nv
from nvfp4_block_scaled_gemv_gb300 import build as libbuild
from nvfp4_block_scaled_gemv_gb300 import layer

P = 256  # a pointer that no case below dereferences


@pytest.fixture(scope="module")
def lib():
    libbuild.build()
    return nv.library()


def moe_ffn(lib, T=4, k=2, E=8, D=64, F=64, size=1 << 40, **opt):
    o = layer._MoeOptions(**(dict(encode_x=1.0, encode_h=1.0, activation=2) | opt))
    return lib.nvfp4_moe_ffn(P, 1, 0, P, P, P, P, P, P, T, k, E, D, F, ctypes.byref(o), P, P, size, None)


@pytest.mark.parametrize("value", [-1, 2])
def test_moe_ffn_refuses_other_roundings(lib, value):
    assert moe_ffn(lib, round_outputs=value) == nv.ERR_INVALID_VALUE


def test_moe_ffn_workspace_holds_32_bit_outputs(lib):
    """Whatever the number of choices, the rows of outputs that the products fill."""
    for T, k, E, D in ((40, 2, 8, 64), (4096, 8, 64, 4096)):
        need = nv.nvfp4_moe_ffn_workspace_bytes(T, k, E, D, 64)
        assert need >= 4 * T * k * D
        assert moe_ffn(lib, T, k, E, D, size=need - 1) == nv.ERR_INVALID_VALUE
