"""The example layer's training step with its routing and its loss (norm, routing,
dispatch, ragged products, gated activation, combine, cross entropy, and all their
gradients) against torch autograd in fp32, and captured into a graph."""
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


@pytest.mark.parametrize("shape", [(37, 512, 256, 4, 2), (300, 1024, 384, 8, 2), (5, 256, 128, 16, 1),
                                   (513, 256, 128, 64, 6)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("vocabulary", [333, 5000])
def test_step_matches_autograd(layer, shape, vocabulary):
    err = layer.run(*shape, vocabulary=vocabulary)
    # the loss: logits of bf16 operands known to 2^-8 each, of a few units, against a loss of
    # log(V) > 5; the head's gradient: its two operands, the rows of out and p, to 2^-8 each and
    # p by what its logits are off
    assert err["loss"] <= 4 * 2.0 ** -8
    assert err["d_head"] <= 8 * 2.0 ** -8
    # through the products from the 8-bit checkpoint (2^-4 / sqrt(3) of each value on average)
    for k in ("dx", "d_norm", "d_router", "dw1", "dw2"):
        assert err[k] <= 2 * 2.0 ** -4 / 3 ** 0.5, (k, err)


def test_step_in_a_graph(layer):
    T, top_k = 130, 2
    w = layer.Weights(512, 256, 8, vocabulary=700)
    x, r = (torch.randn(T, 512, device="cuda").to(layer.BF16) for _ in range(2))
    y = torch.randint(0, 700, (T,), device="cuda").to(torch.int32)
    layer.train_step(w, x, r, y, top_k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.train_step(w, x, r, y, top_k)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss, out, grads = layer.train_step(w, x, r, y, top_k)
    # other tokens, which choose other experts: the graph follows
    x.copy_(torch.randn(T, 512, device="cuda"))
    y.copy_(torch.randint(0, 700, (T,), device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    want_loss, want_out, want = layer.train_step(w, x, r, y, top_k)
    assert torch.equal(loss, want_loss) and torch.equal(out, want_out)
    assert all(torch.equal(grads[k], want[k]) for k in want)
