"""The cross entropy where its values are known more closely than loss_ref.py's bounds
say: whole-number logits, tokens that are nearly certain, far logits."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import loss_ref as L
from tests.test_gpu_loss import BF16, backward, check_backward, check_forward, forward, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    assert dg.get_device_status() == 0


def whole(T, V, K, seed, words=3):
    """Operands of small whole numbers, so that every sum of their products is exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randint(-2, 3, (T, K), generator=g, device="cuda").to(BF16)
    W = torch.randint(-words, words + 1, (V, K), generator=g, device="cuda").to(BF16)
    return X, W


@pytest.mark.parametrize("shape", [(40, 3000, 256), (300, 3000, 256), (7, 20000, 1024), (500, 1500, 1024), (9, 1, 64),
                                   (130, 1, 64), (70, 2, 8)], ids=lambda s: "x".join(map(str, s)))
def test_losses_of_exact_logits(shape):
    # The loss by itself is off by what its exponentials (2^-21 of each, as everywhere), the
    # sums (V / 64 and 32 terms) and its logarithm are, relative to the loss or to the one that
    # the target's exponential is; not by a rounding of lse, which may be hundreds.
    T, V, K = shape
    X, W = whole(T, V, K, seed=K)
    z = L.logits(X, W)
    assert z.abs().max() < 2 ** 24
    for t in (z.argmax(1), z.argsort(1)[:, V // 2], z.argmin(1)):
        t = t.to(torch.int32)
        loss, _ = forward(X, W, t)
        want = L.loss(X, W, t)[0]
        # (a log2 of the sum: off by 2 ulp, below 2^-22 of its value, which is at most 2 want + 2)
        lim = 2.0 ** -21 * (1 + V / 2 ** 14) + 2.0 ** -21 * want
        assert (loss >= 0).all(), loss.min()
        assert ((loss.double() - want).abs() <= lim).all(), (loss.double() - want).abs().max()


def certain(T, V, K, z, seed):
    """Tokens whose targets' logits are near z, those of the other words a few units: each with
    a target of its own, along whose row its own points."""
    X, W, _, d = inputs(T, V, K, seed, ignored=0.0)
    t = torch.arange(T, device="cuda") * (V // T)
    x = X.double()
    W[t] = (x * (z / x.square().sum(1, keepdim=True))).to(BF16)
    return X, W, t.to(torch.int32), d


@pytest.mark.parametrize("shape", [(200, 3000, 7168, 17.0), (40, 3000, 7168, 17.0), (300, 3000, 2048, 14.0)],
                         ids=lambda s: "x".join(map(str, s)))
def test_gradients_of_tokens_that_are_nearly_certain(shape):
    # p at the target is -(1 - s) with 1 - s near 1e-3, so that an error e of the logit is one
    # of e / 1e-3 of p.  A sum of K / 16 steps in the tensor cores drops half of 2^-23 of its
    # partial sum at each; of 32 steps at a time, added up in fp32, that is less than 1e-6 of the logit
    # (32 / 2 2^-23 / 2: half of the steps' partial sum on average).  Then the exponential and its
    # argument (2^-20 of s), p's and the output's roundings to bf16.
    T, V, K, z = shape
    X, W, t, d = certain(T, V, K, z, seed=5)
    loss, lse = forward(X, W, t)
    check_forward(X, W, t, loss, lse)
    p = L.probabilities(X, W, t, lse, torch.ones_like(d))
    rest = -p[torch.arange(T), t.long()]
    assert 1e-4 < rest.min() and rest.max() < 0.05
    dX, dW = backward(X, W, t, lse, d)
    check_backward(X, W, t, lse, d, dX, dW)
    p = p * d.double()[:, None]
    e = (1e-6 * z + 2.0 ** -20) / rest     # of p at each target
    far = 2 * L.BF16_ROUND
    at = t.long()
    want = p.t() @ X.double()
    off = (dW.double() - want)[at]
    assert (off.norm(dim=1) <= (e + far) * want[at].norm(dim=1) * 1.02).all(), (off.norm(dim=1) / want[at].norm(dim=1)).max()
    want = p @ W.double()
    lim = far * want.norm(dim=1) + e * p[torch.arange(T), at].abs() * W[at].double().norm(dim=1)
    off = (dX.double() - want).norm(dim=1)
    assert (off <= 1.02 * lim + far * p.abs().amax(1) * 1e-3).all(), (off / lim).max()


@pytest.mark.parametrize("T", [40, 300])
@pytest.mark.parametrize("words", [3, 40])
def test_gradients_of_exact_logits(T, words):
    # logits of hundreds to thousands, one word has it all or two share it: p is off by the
    # rounding of log2(e) lse (2^-24 of it, times ln 2), the fused multiply-add's (2^-24 of its result,
    # at most a few hundred where the exponential is not 0) and 2^-21
    V, K = 3000, 256
    X, W = whole(T, V, K, seed=words, words=words)
    z = L.logits(X, W)
    t = torch.where(torch.arange(T, device="cuda") % 3 == 0, z.argmax(1), z.argsort(1)[:, V - 2]).to(torch.int32)
    d = torch.randn(T, device="cuda")
    lse = torch.logsumexp(z, 1).float()
    dX, dW = backward(X, W, t, lse, d)
    p = L.probabilities(X, W, t, lse, d)
    s = torch.exp(z - lse.double()[:, None])
    e = 2.0 ** -24 * (lse.double().abs()[:, None] + 130) + 2.0 ** -21
    off = e * s * d.double().abs()[:, None] + L.BF16_ROUND * p.abs()
    for got, want, mag, err in ((dX, p @ W.double(), p.abs() @ W.double().abs(), off @ W.double().abs()),
                                (dW, p.t() @ X.double(), p.t().abs() @ X.double().abs(), off.t() @ X.double().abs())):
        lim = L.BF16_ROUND * (1 + L.BF16_ROUND) * want.abs() + 1e-5 * mag + 1.01 * err + 1e-30
        assert ((got.double() - want).abs() <= lim).all(), ((got.double() - want).abs() - lim).max()


def test_far_logits():
    # as test_flat_and_peaked's farthest, with a bound: the logits' own error is large, and p's
    # follows it as far as e^e - 1 <= 2 e goes (e < 1.2)
    X, W, t, d = inputs(90, 3001, 128, seed=3, scale=2000.0)
    e, es = L.slack(X, W)
    assert (e + es).max() < 1.2
    loss, lse = forward(X, W, t)
    check_backward(X, W, t, lse, d, *backward(X, W, t, lse, d))


def test_rows_of_the_output_matrix_that_share_a_component():
    # a token's p sum to 0 but for their rounding to bf16, which the shared component multiplies
    X, W, t, d = inputs(150, 4000, 512, seed=11, ignored=0.1)
    W = (W.float() + 3.0 * torch.randn(512, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
         * 512 ** -0.5).to(BF16)
    loss, lse = forward(X, W, t)
    check_forward(X, W, t, loss, lse)
    check_backward(X, W, t, lse, d, *backward(X, W, t, lse, d))


def test_a_vocabulary_of_many_pieces():
    # sums over 2^20 words at most, in 8 shares at least: 8192 steps of the tensor cores, each of
    # which drops 2^-23 of its partial sum at most, 1e-3 in all; p's rounding and the output's
    T, V, K = 3, 200_000_000, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    W = torch.empty(V, K, dtype=BF16, device="cuda").normal_(0.0, 0.7, generator=g)
    t = torch.tensor([V - 1, 5, 2 ** 27 + 3], dtype=torch.int32, device="cuda")
    d = torch.tensor([1.0, -0.5, 0.25], device="cuda")
    loss, lse = forward(X, W, t)
    z = torch.cat([L.logits(X, w) for w in W.split(25_000_000)], 1)
    want = torch.logsumexp(z, 1)
    assert ((lse.double() - want).abs() <= 1e-6 * want).all()
    dX, dW = backward(X, W, t, lse, d)
    p = torch.exp(z.sub_(lse.double()[:, None]))
    p[torch.arange(T), t.long()] -= 1.0
    p *= d.double()[:, None]
    want = sum(p[:, i:i + 25_000_000] @ W[i:i + 25_000_000].double() for i in range(0, V, 25_000_000))
    assert ((dX.double() - want).norm(dim=1) <= (2 * L.BF16_ROUND + 1e-3) * want.norm(dim=1)).all()
    for rows in (slice(0, 300), slice(2 ** 27 - 100, 2 ** 27 + 200), slice(V - 300, V)):
        want = p[:, rows].t() @ X.double()
        assert (dW[rows].double() - want).norm() <= 2 * L.BF16_ROUND * want.norm()
