"""Softmax cross entropy of a product over a vocabulary, and its gradients, against
the definition in 64 bits (bounds: loss_ref.py)."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import loss_ref as L
from tests.launches import launched

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
KEEP = -7.0   # what no call may write


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    assert dg.get_device_status() == 0


def inputs(T, V, K, seed, ignored=0.2, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    W = (torch.randn(V, K, generator=g, device="cuda") * scale * K ** -0.5).to(BF16)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    skip = torch.rand(T, generator=g, device="cuda") < ignored
    t = torch.where(skip, torch.where(t % 2 == 0, -1, V), t).to(torch.int32)
    return X, W, t, torch.randn(T, generator=g, device="cuda")


def guarded(*shape, dtype=BF16):
    """A tensor with rows behind it that nothing may touch."""
    x = torch.full((shape[0] + 3, *shape[1:]), KEEP, dtype=dtype, device="cuda")
    return x[:shape[0]], x[shape[0]:]


def workspace(n):
    return torch.full((max(n, 16) + 64,), 0xFF, dtype=torch.uint8, device="cuda")


def forward(X, W, t, stream=None):
    (T, K), V = X.shape, W.shape[0]
    n = dg.linear_cross_entropy_workspace_bytes(T, V, K)
    work = workspace(n)
    (loss, lg), (lse, sg) = guarded(T, dtype=torch.float32), guarded(T, dtype=torch.float32)
    dg.linear_cross_entropy(X, W, t, loss, lse, work, n, T, V, K, stream=stream)
    torch.cuda.synchronize()
    assert (lg == KEEP).all() and (sg == KEEP).all() and (work[n:] == 0xFF).all()
    return loss, lse


def backward(X, W, t, lse, d, want_x=True, want_w=True, stream=None):
    (T, K), V = X.shape, W.shape[0]
    n = dg.linear_cross_entropy_backward_workspace_bytes(T, V, K)
    work = workspace(n)
    (dX, xg), (dW, wg) = guarded(T, K), guarded(V, K)
    dg.linear_cross_entropy_backward(X, W, t, lse, d, dX if want_x else None, dW if want_w else None, work, n, T,
                                     V, K, stream=stream)
    torch.cuda.synchronize()
    assert (xg == KEEP).all() and (wg == KEEP).all() and (work[n:] == 0xFF).all()
    return dX, dW


def check_forward(X, W, t, loss, lse):
    want, want_lse = L.loss(X, W, t)
    e, es = L.slack(X, W)
    assert ((lse.double() - want_lse).abs() <= es).all(), (lse.double() - want_lse).abs().max()
    lim = torch.where(L.there(t, W.shape[0]), e + es + 2 * L.U * want.abs(), 0.0)
    assert ((loss.double() - want).abs() <= lim).all(), (loss.double() - want).abs().max()


def check_backward(X, W, t, lse, d, dX, dW):
    p = L.probabilities(X, W, t, lse, d)
    e, es = L.slack(X, W)
    # each p: a relative error of its exponential, its rounding; (s - 1 is off by what s is)
    s = (p / d.double()[:, None].where(d[:, None] != 0, 1.0)).abs()
    at = L.there(t, W.shape[0]).nonzero()[:, 0]
    s[at, t[at].long()] = 1.0
    off = s * d.double().abs()[:, None] * (2 * (e + es) + 2.0 ** -20)[:, None] + L.BF16_ROUND * p.abs()
    off = torch.where(L.there(t, W.shape[0])[:, None], off, 0.0)
    for name, got, want, mag, err in (
            ("dX", dX, p @ W.double(), p.abs() @ W.double().abs(), off @ W.double().abs()),
            ("dW", dW, p.t() @ X.double(), p.t().abs() @ X.double().abs(), off.t() @ X.double().abs())):
        lim = L.BF16_ROUND * (1 + L.BF16_ROUND) * want.abs() + 1e-5 * mag + err * 1.01 + 1e-38
        bad = ~((got.double() - want).abs() <= lim)
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist())


SHAPES = [(1, 1, 8), (1, 1000, 256), (3, 17, 8), (61, 130, 64), (128, 128, 128), (130, 2051, 264), (257, 513, 72),
          (40, 32003, 512), (700, 5000, 136), (2000, 5000, 264), (300, 257, 1032), (2, 50003, 2048)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_loss_and_gradients(shape):
    T, V, K = shape
    X, W, t, d = inputs(T, V, K, seed=T + V)
    loss, lse = forward(X, W, t)
    check_forward(X, W, t, loss, lse)
    dX, dW = backward(X, W, t, lse, d)
    check_backward(X, W, t, lse, d, dX, dW)
    # either gradient alone
    assert torch.equal(backward(X, W, t, lse, d, want_w=False)[0], dX)
    assert torch.equal(backward(X, W, t, lse, d, want_x=False)[1], dW)


@pytest.mark.parametrize("shape", [(12300, 20001, 64), (6000, 40011, 256), (50000, 4097, 8)],
                         ids=lambda s: "x".join(map(str, s)))
def test_pieces_of_the_vocabulary(shape):
    T, V, K = shape
    assert dg.linear_cross_entropy_backward_workspace_bytes(T, V, K) < 2 * T * V   # more than one piece
    X, W, t, d = inputs(T, V, K, seed=1)
    pieces = -(-V // max(4096, (384 << 20) // (2 * T)))
    words = -(-(-(-V // pieces)) // 256) * 256
    t[0], t[1], t[2], t[3] = V - 1, words, words - 1, 0    # (at the borders)
    loss, lse = forward(X, W, t)
    check_forward(X, W, t, loss, lse)
    check_backward(X, W, t, lse, d, *backward(X, W, t, lse, d))


def test_no_target_at_all():
    X, W, t, d = inputs(20, 300, 64, seed=2)
    t[:] = -1
    d[:] = float("nan")   # (not read)
    loss, lse = forward(X, W, t)
    check_forward(X, W, t, loss, lse)
    assert (loss == 0).all()
    dX, dW = backward(X, W, t, lse, d)
    assert (dX == 0).all() and (dW == 0).all()


def test_no_tokens():
    X, W, t, d = inputs(0, 300, 64, seed=2)
    dX, dW = backward(X, W, t, d, d)
    assert (dW == 0).all()
    dg.linear_cross_entropy(None, W, None, None, None, None, 0, 0, 300, 64)


@pytest.mark.parametrize("scale", [0.0, 30.0, 2000.0])
def test_flat_and_peaked(scale):
    # all logits equal; logits of a hundred, of thousands (one word has it all)
    X, W, t, d = inputs(90, 3001, 128, seed=3, scale=scale)
    loss, lse = forward(X, W, t)
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all()
    check_forward(X, W, t, loss, lse)
    dX, dW = backward(X, W, t, lse, d)
    assert torch.isfinite(dX).all() and torch.isfinite(dW).all()
    if scale <= 30.0:
        check_backward(X, W, t, lse, d, dX, dW)


def test_one_output_only():
    X, W, t, _ = inputs(70, 900, 64, seed=4)
    loss, lse = forward(X, W, t)
    n = dg.linear_cross_entropy_workspace_bytes(70, 900, 64)
    for i, want in ((0, loss), (1, lse)):
        out = torch.zeros(70, device="cuda")
        args = (out, None) if i == 0 else (None, out)
        dg.linear_cross_entropy(X, W, t, *args, workspace(n), n, 70, 900, 64)
        assert torch.equal(out, want)


def test_streams_graphs_and_limits():
    T, V, K = 300, 20000, 512
    X, W, t, d = inputs(T, V, K, seed=5)
    loss, lse = forward(X, W, t)
    dX, dW = backward(X, W, t, lse, d)
    want = [x.clone() for x in (loss, lse, dX, dW)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (*forward(X, W, t, stream=side), *backward(X, W, t, lse, d, stream=side))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    nf, nb = (f(T, V, K) for f in (dg.linear_cross_entropy_workspace_bytes,
                                   dg.linear_cross_entropy_backward_workspace_bytes))
    work = workspace(max(nf, nb))
    outs = [torch.zeros_like(x) for x in want]

    def both(stream=None):
        dg.linear_cross_entropy(X, W, t, outs[0], outs[1], work, nf, T, V, K, stream=stream)
        dg.linear_cross_entropy_backward(X, W, t, outs[1], d, outs[2], outs[3], work, nb, T, V, K, stream=stream)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # new inputs through the same graph
    X2, W2, t2, d2 = inputs(T, V, K, seed=6)
    for a, b in zip((X, W, t, d), (X2, W2, t2, d2)):
        a.copy_(b)
    g.replay()
    torch.cuda.synchronize()
    check_forward(X, W, t, outs[0], outs[1])
    check_backward(X, W, t, outs[1], d, outs[2], outs[3])
    for sms in (1, 3, 132):
        dg.set_num_sms(sms)
        try:
            for o in outs:
                o.zero_()
            both()
            torch.cuda.synchronize()
            assert all(b <= sms for b, _, _ in launched(both))
        finally:
            dg.set_num_sms(0)
        check_forward(X, W, t, outs[0], outs[1])
        check_backward(X, W, t, outs[1], d, outs[2], outs[3])


@pytest.mark.parametrize("plan", [(True, 256, 256, 1), (True, 256, 192, 1), (True, 256, 224, 2), (True, 256, 256, 2), (True, 256, 256, 4), (False, 64, 64, 1),
                                  (False, 64, 64, 8), (False, 128, 64, 2), (False, 192, 64, 4),
                                  (False, 256, 128, 1), (False, 128, 128, 3), (False, 256, 128, 8)],
                         ids=lambda p: "x".join(str(int(v)) for v in p))
@pytest.mark.parametrize("shape", [(200, 3001, 264), (61, 700, 1024), (50000, 4500, 72)],
                         ids=lambda s: "x".join(map(str, s)))
def test_every_tiling(plan, shape):
    X, W, t, d = inputs(*shape, seed=9)
    dg.debug_force_ragged_plan(*plan)
    try:
        loss, lse = forward(X, W, t)
        dX, dW = backward(X, W, t, lse, d)
    finally:
        dg.debug_force_ragged_plan()
    check_forward(X, W, t, loss, lse)
    check_backward(X, W, t, lse, d, dX, dW)


def test_a_mean_loses_no_precision():
    # the same d_loss for all tokens, no power of two: p is rounded near -1, not near -d
    X, W, t, _ = inputs(45, 20000, 256, seed=7, ignored=0.0)
    d = torch.full((45,), 1 / 45.35, device="cuda")
    loss, lse = forward(X, W, t)
    dX, dW = backward(X, W, t, lse, d)
    for got, want in zip((dX, dW), L.gradients(X, W, t, lse, d)):
        # a rounding to bf16 is uniform in half a step, a step 2^-7 of values from 1 to 2: at most
        # 2^-8 / sqrt(3) of them in the mean square; p's own rounding, of single words' small shares
        # and by 2^-9 of the -1's, adds less than half of that
        assert (got.double() - want).norm() <= 1.2 * 2.0 ** -8 / 3 ** 0.5 * want.norm()


def test_forced_tilings_that_the_products_lack_are_refused():
    X, W, t, d = inputs(20, 300, 64, seed=2)
    for plan in ((False, 144, 64, 1), (False, 128, 48, 1)):
        dg.debug_force_ragged_plan(*plan)
        try:
            with pytest.raises(dg.DGError) as e:
                forward(X, W, t)
        finally:
            dg.debug_force_ragged_plan()
        assert e.value.status == 2


@pytest.mark.parametrize("T", [5, 100])
def test_deep_reductions_lose_no_precision(T):
    # the tensor cores' sums drop bits at each of their 448 steps here (2.2e-6 of the loss in all);
    # 32 of them at a time, added up in fp32: a step drops half of 2^-23 of its partial sum on
    # average, the 14 partial sums, half as large on the way, come to sqrt(14) times their total:
    # 32 / 2 2^-23 / 2 sqrt(14) / 4 < 1e-6
    X, W, t, _ = inputs(T, 3000, 7168, seed=3, ignored=0.0)
    loss, lse = forward(X, W, t)
    want, want_lse = L.loss(X, W, t)
    for got, ref in ((loss, want), (lse, want_lse)):
        assert (got.double() - ref).norm() <= 1e-6 * ref.norm()


def test_operands_past_32_bits():
    # 2.4e9 elements of W and of dW; the words of interest at both ends
    T, V, K = 3, 300000, 8008
    assert V * K > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.randn(T, K, generator=g, device="cuda").to(BF16)
    W = torch.empty(V, K, dtype=BF16, device="cuda").normal_(0.0, 2 * K ** -0.5, generator=g)
    t = torch.tensor([V - 1, 0, 270000], dtype=torch.int32, device="cuda")
    d = torch.tensor([1.0, -0.5, 0.25], device="cuda")
    loss, lse = forward(X, W, t)
    z = torch.cat([L.logits(X, w) for w in W.split(20000)], 1)
    want = torch.logsumexp(z, 1)
    assert ((lse.double() - want).abs() <= 2e-5 * want).all()
    hit = z.gather(1, t.long()[:, None])[:, 0]
    assert ((loss.double() - (want - hit)).abs() <= 2e-5 * want).all()
    dX, dW = backward(X, W, t, lse, d)
    p = torch.exp(z - lse.double()[:, None])
    p[torch.arange(3), t.long()] -= 1.0
    p *= d.double()[:, None]
    wx = sum(p[:, i:i + 20000] @ W[i:i + 20000].double() for i in range(0, V, 20000))
    assert (dX.double() - wx).norm() <= 2 * L.BF16_ROUND * wx.norm()
    for rows in (slice(0, 300), slice(269900, 270100), slice(V - 300, V)):
        ww = p[:, rows].t() @ X.double()
        assert (dW[rows].double() - ww).norm() <= 2 * L.BF16_ROUND * ww.norm()


def test_waits_that_run_out():
    # the loads switched off: the waits give up, which is reported, and nothing is stored
    X, W, t, d = inputs(300, 2000, 256, seed=2)
    n = dg.linear_cross_entropy_backward_workspace_bytes(300, 2000, 256)
    work, lse = workspace(n), forward(X, W, t)[1]
    dX, dW = torch.full_like(X, KEEP), torch.full_like(W, KEEP)
    dg.set_wait_timeout_ns(2_000_000)
    dg.debug_set_skip_producer(True)
    try:
        dg.linear_cross_entropy_backward(X, W, t, lse, d, dX, dW, work, n, 300, 2000, 256)
        torch.cuda.synchronize()
        assert dg.get_device_status() == 7
        dg.linear_cross_entropy(X, W, t, torch.empty(300, device="cuda"), lse, work, n, 300, 2000, 256)
        torch.cuda.synchronize()
        assert dg.get_device_status() == 7
    finally:
        dg.debug_set_skip_producer(False)
        dg.set_wait_timeout_ns(0)
    assert (dW == KEEP).all()
    # and the next call is whole again
    loss, lse = forward(X, W, t)
    check_forward(X, W, t, loss, lse)
    check_backward(X, W, t, lse, d, *backward(X, W, t, lse, d))


def test_two_calls_at_once():
    # on two streams, each with a workspace of its own
    a, b = inputs(500, 9000, 512, seed=1), inputs(33, 30000, 256, seed=2)
    want = []
    for X, W, t, d in (a, b):
        loss, lse = forward(X, W, t)
        want.append((loss, lse, *backward(X, W, t, lse, d)))
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for X, W, t, d in (a, b):
        T, V, K = X.shape[0], W.shape[0], X.shape[1]
        n = max(dg.linear_cross_entropy_workspace_bytes(T, V, K),
                dg.linear_cross_entropy_backward_workspace_bytes(T, V, K))
        outs.append((torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(X),
                     torch.empty_like(W), workspace(n), n))
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (X, W, t, d), (loss, lse, dX, dW, work, n) in zip(streams, (a, b), outs):
            T, V, K = X.shape[0], W.shape[0], X.shape[1]
            dg.linear_cross_entropy(X, W, t, loss, lse, work, n, T, V, K, stream=s)
            dg.linear_cross_entropy_backward(X, W, t, lse, d, dX, dW, work, n, T, V, K, stream=s)
    torch.cuda.synchronize()
    for got, ref in zip(outs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, ref))
