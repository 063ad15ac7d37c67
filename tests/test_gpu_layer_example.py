"""The example layer runs the operators together, and stays as near its fp32 form as 4-bit
activations allow."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

import nvfp4_block_scaled_gemv_gb300 as nv  # noqa: E402
from nvfp4_block_scaled_gemv_gb300 import build as libbuild  # noqa: E402

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    libbuild.build()
    nv.library()


@pytest.mark.parametrize("tokens", [1, 64, 700])
def test_example_layer(tokens):
    import moe_layer

    # E2M1 with a scale per 16 elements leaves ~10% of an activation's size as noise (a
    # step is a sixth to a third of the value); it passes two products and a gate
    assert moe_layer.main(tokens) < 0.25
    assert nv.nvfp4_tensor_wait_timeouts(reset=True) == 0


def test_example_layer_repeats_bit_for_bit():
    import moe_layer

    layer = moe_layer.Layer()
    x = torch.randn(300, 512, device="cuda:0").bfloat16()
    first = layer(x)
    assert all(torch.equal(layer(x), first) for _ in range(3))
