"""The 64-bit definitions the GPU tests compare with: their gradients against
central differences of their forward passes (no GPU)."""
import pytest
import torch

from tests import operators_ref as R

F64 = torch.float64


def differences(f, x, dy, at, h=1e-6):
    """d/dx[at] of sum(f(x) * dy), by central differences."""
    got = []
    for i in at:
        lo, hi = x.clone(), x.clone()
        lo.view(-1)[i] -= h
        hi.view(-1)[i] += h
        got.append(((f(hi) - f(lo)) * dy).sum() / (2 * h))
    return torch.stack(got)


def draw(*shape, seed=0, scale=1.0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64) * scale


@pytest.mark.parametrize("M,K", [(1, 128), (3, 256)])
def test_norm_gradient(M, K):
    x, r, w, dy = draw(M, K, seed=1), draw(M, K, seed=2), draw(K, seed=3), draw(M, K, seed=4)
    eps = 1e-3
    h, rstd, _ = R.norm(x, r, w, eps)
    dx, dw = R.norm_backward(dy, h, rstd, w, None)
    at = list(range(0, M * K, 37))
    want = differences(lambda t: R.norm(t, r, w, eps)[2], x, dy, at)
    assert torch.allclose(dx.view(-1)[at], want, rtol=1e-6, atol=1e-7)
    want = differences(lambda t: R.norm(x, r, t, eps)[2], w, dy, at[:5])
    assert torch.allclose(dw[at[:5]], want, rtol=1e-6, atol=1e-7)
    dr = draw(M, K, seed=5)
    assert torch.equal(R.norm_backward(dy, h, rstd, w, dr)[0], dx + dr)


def test_swiglu_gradient():
    gu, dy = draw(3, 256, seed=6, scale=3.0), draw(3, 128, seed=7)
    at = list(range(0, 768, 41))
    want = differences(R.swiglu, gu, dy, at)
    assert torch.allclose(R.swiglu_backward(gu, dy).view(-1)[at], want, rtol=1e-6, atol=1e-8)


def test_product_gradients():
    sizes = [3, 0, 5]
    x, w = draw(8, 16, seed=8), draw(3, 24, 16, seed=9)
    dy = draw(8, 24, seed=10)
    f = lambda a, b: R.products("nt", a, b, sizes)[0]
    dx = R.products("nn", dy, w, sizes)[0]
    dw = R.products("tn", dy, x, sizes)[0]
    assert dw.shape == w.shape and torch.all(dw[1] == 0)
    at = list(range(0, 128, 17))
    assert torch.allclose(dx.view(-1)[at], differences(lambda t: f(t, w), x, dy, at), rtol=1e-6,
                          atol=1e-8)
    at = list(range(0, 24 * 16 * 3, 97))
    assert torch.allclose(dw.view(-1)[at], differences(lambda t: f(x, t), w, dy, at), rtol=1e-6,
                          atol=1e-8)


def test_packed_scales_unpack():
    words = torch.zeros(2, 4, dtype=torch.int32)
    b = words.view(torch.uint8).view(2, 4, 4)
    for g in range(6):
        for m in range(3):
            b[g // 4, m, g % 4] = 100 + 10 * g + m
    got = R.unpack_ue8m0(words, 3, 6)
    want = torch.tensor([[2.0 ** (100 + 10 * g + m - 127) for g in range(6)] for m in range(3)],
                        dtype=F64)
    assert torch.equal(got, want)
