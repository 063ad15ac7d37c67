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


@pytest.mark.parametrize("T,k,E,D,F", [(1, 8, 256, 7168, 2048), (128, 8, 256, 7168, 2048), (64, 16, 1024, 4096, 1024),
                                       (500, 4, 37, 2048, 512), (4096, 8, 64, 4096, 2048)])
def test_moe_ffn_workspace_holds_tiles_of_outputs_and_no_scale_atoms_of_them(lib, T, k, E, D, F):
    """Rows of outputs for the choices and for one tile's rest per expert, not the 128 rows that
    a tile's scales take."""
    s = nv.nvfp4_moe_shape(T, k, E)
    outputs = 4 * D * (T * k + s["tile_rows"] * min(E, T * k))
    codes = s["row_capacity"] * ((D + F) // 2 + -(-D // 64) * 4 + -(-F // 64) * 4)
    need = nv.nvfp4_moe_ffn_workspace_bytes(T, k, E, D, F)
    assert need <= outputs + codes + s["plan_bytes"] + 4 * T * k + 8 * E + 9 * 256


@pytest.mark.parametrize("T,k,E,D,F", [(4, 2, 8, 48, 64), (4, 2, 8, 64, 48), (4, 2, 8, 0, 64), (4, 2, 8, 64, 0),
                                       (4, 2, 8, -64, 64), (4, 9, 8, 64, 64), (4, 2, 8, 1 << 30, 1 << 30),
                                       (1 << 22, 4, 64, 1 << 20, 64), (4, 2, 8, 64, 1 << 31)])
def test_moe_ffn_workspace_of_sizes_that_are_refused_is_0(lib, T, k, E, D, F):
    assert nv.nvfp4_moe_ffn_workspace_bytes(T, k, E, D, F) == 0
    assert moe_ffn(lib, T, k, E, D, F) in (nv.ERR_INVALID_VALUE, nv.ERR_UNSUPPORTED_SHAPE)


SM_SMEM, RESERVED = 228 * 1024, 1024  # shared memory of an SM, and what every CTA takes beside its own


def footprints(lib):
    """{(rows of a product's tile, gated): (shared memory, columns of tensor memory)}."""
    fn = lib["_ZN5nvfp417product_footprintEib"]
    fn.argtypes, fn.restype = [ctypes.c_int, ctypes.c_bool], ctypes.c_uint64
    both = {(rows, gated): fn(rows, gated) for rows in (16, 32, 64, 128, 256) for gated in (False, True)}
    return {key: (v & 0xFFFFFFFF, v >> 32) for key, v in both.items()}


def blockdot_footprint(lib):
    """The least shared memory of the block-dot kernel's CTA, and its columns."""
    fn = lib["_ZN5nvfp419blockdot_smem_bytesEbiii"]
    fn.argtypes, fn.restype = [ctypes.c_bool] + [ctypes.c_int] * 3, ctypes.c_size_t
    return min(fn(permuted, blocks, 8, stages) for permuted in (False, True) for blocks in (1, 2)
               for stages in (1, 2, 32)), 256


def test_tensor_memory_is_never_asked_for_beyond_an_sm(lib):
    """Whatever CTAs of products, of the tensor-core GEMV and of the block-dot kernel share an SM
    between streams: one that waited for columns there could, in a cluster, hold up another
    SM's for ever."""
    # the GEMV's stages: an A tile of 128 x 128 bytes, a B tile of 16 x 128 and eight scale atoms;
    # and 2 KB (the ranks' sums of one vector, the alignment)
    gemv = [(s * (128 * 128 + 16 * 128 + 8 * 512) + 2048, c) for s, c in ((2, 128), (4, 256))]
    kinds = list(footprints(lib).values()) + gemv
    kinds.append(blockdot_footprint(lib))
    assert all(smem <= 227 * 1024 for smem, _ in kinds)
    for first in kinds:
        packed = [(first,)]
        while packed:
            ctas = packed.pop()
            assert sum(columns for _, columns in ctas) <= 512, ctas
            room = SM_SMEM - sum(smem + RESERVED for smem, _ in ctas)
            packed += [ctas + (k,) for k in kinds if k[0] + RESERVED <= room]


def test_calls_say_what_they_do_with_signs():
    for call in (nv.gemm, nv.nvfp4_gemm):
        assert "signs" in call.__doc__ and "ignored" in call.__doc__
