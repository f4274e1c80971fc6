"""The example layer (norm, ragged products, gated activation with its 8-bit
checkpoint, masked FP8 GEMMs) against torch autograd in fp32."""
import importlib.util
import os

import pytest
import torch

from moe_grouped_gemm_bf16_gb300 import _build

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    _build.build()
    torch.cuda.init()
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("shape", [(37, 512, 256, 4, 2), (300, 1024, 384, 8, 2), (5, 256, 128, 16, 1)],
                         ids=lambda s: "x".join(map(str, s)))
def test_layer_matches_autograd(layer, shape):
    err = layer.run(*shape)
    # bf16 values between the operators: up to 2^-8 of themselves each, a chain of
    # four; the checkpoint and FP8 operands: codes are off by 2^-4 of themselves
    # at most, 2^-4 / sqrt(3) on average, two of them in a product
    assert err["out"] <= 4 * 2.0 ** -8
    for k in ("dx", "d_norm", "dw1", "dw2"):
        assert err[k] <= 2 * 2.0 ** -4 / 3 ** 0.5, (k, err)
    # four roundings to 8 bits in the decoding step (two operands, twice)
    assert err["decode"] <= 4 * 2.0 ** -4 / 3 ** 0.5, err
