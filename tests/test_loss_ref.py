"""The definition that the cross entropy is tested against: its gradients against
differences."""
import torch

from tests import loss_ref as L


def test_gradients_against_differences():
    g = torch.Generator().manual_seed(0)
    X, W = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((4, 6), (9, 6)))
    t, d = torch.tensor([3, -1, 8, 9]), torch.randn(4, generator=g, dtype=torch.float64)
    value = lambda X, W: (L.loss(X, W, t)[0] * d).sum()
    loss, lse = L.loss(X, W, t)
    assert loss[1] == 0 and loss[3] == 0 and (loss[[0, 2]] > 0).all()
    for got, x, f in zip(L.gradients(X, W, t, lse, d), (X, W), (lambda x: value(x, W), lambda x: value(X, x))):
        for i in range(x.numel()):
            h = torch.zeros(x.numel(), dtype=torch.float64)
            h[i] = 1e-6
            h = h.view(x.shape)
            assert abs((f(x + h) - f(x - h)) / 2e-6 - got.flatten()[i]) < 1e-8
