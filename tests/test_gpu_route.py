"""Routing of tokens to experts and its gradient against the definition in 64 bits.

Bounds.  u = 2^-24.  The choice is exact.  A weight: expf is off by 2 ulp at most
(4 u), its argument's rounding by |x - max| u, the sum of n terms by n u, the
quotients and the scale by u each: (16 + |x - max| + n) u of itself, n = 32 for the
lanes' partial sums and the tree.  A gradient's terms: twice that of the sum over
magnitudes, and the rounding to bf16 where the logits are.  Below 2^-126 an fp32
value is a multiple of 2^-149: an exponential, a quotient and the scale round by half
of it or less each (expf by 2 ulp), 4 2^-149 of error in all."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import moe_ref as M
from tests.launches import launched

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 4 * 2.0 ** -149


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    assert dg.get_device_status() == 0


def logits(T, G, bf16, seed, scale=1.5):
    x = torch.from_numpy(np.random.default_rng(seed).normal(size=(T, G)) * scale).float()
    return x.to(torch.bfloat16) if bf16 else x


def spread(x):
    """|x - max| at most, over what is finite."""
    f = x[np.isfinite(x)]
    return float(f.max() - f.min()) if f.size else 0.0


def within(got, want, lim):
    bad = ~(np.abs(got - want) <= lim)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def run(x, bias, k, sigmoid, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, stream=None):
    T, G = x.shape
    e = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    fn = dg.route_top_k_bf16 if x.dtype == torch.bfloat16 else dg.route_top_k_fp32
    fn(x.cuda(), None if bias is None else bias.cuda(), e, w, T, G, k, sigmoid, groups, top_groups, best,
       renorm, scale, stream=stream)
    torch.cuda.synchronize()
    return e.cpu().numpy(), w.cpu().double().numpy()


def check(x, bias, k, sigmoid, groups=1, top_groups=1, best=1, renorm=True, scale=1.0, tiny=TINY):
    e, w = run(x, bias, k, sigmoid, groups, top_groups, best, renorm, scale)
    xn = x.double().numpy()
    we, ww = M.route(xn, None if bias is None else bias.numpy(), k, sigmoid, groups, top_groups, best, renorm,
                     scale)
    assert np.array_equal(e, we), np.argwhere(e != we)[:5].tolist()
    within(w, ww, (48 + spread(xn)) * U * np.abs(ww) + tiny)


CASES = [  # T, G, k, groups, top_groups, best
    (1, 8, 1, 1, 1, 1), (7, 256, 8, 8, 4, 2), (33, 60, 6, 1, 1, 1), (5, 1, 1, 1, 1, 1), (64, 160, 6, 8, 3, 1),
    (9, 33, 32, 1, 1, 1), (3, 1024, 32, 32, 17, 2), (17, 384, 8, 6, 2, 2), (4, 500, 9, 4, 2, 1),
    (130, 64, 4, 32, 16, 2), (12, 96, 3, 3, 3, 2), (37, 7, 3, 1, 1, 1), (99, 16, 8, 8, 6, 1),
    (50, 32, 5, 4, 2, 2), (1, 24, 8, 3, 2, 2), (35, 64, 16, 16, 7, 2), (2, 48, 11, 12, 5, 2), (6, 30, 10, 3, 3, 1)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c)))
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("biased,renorm", [(True, True), (False, True), (True, False)])
def test_choice_and_weights(case, sigmoid, bf16, biased, renorm):
    T, G, k, groups, top_groups, best = case
    x = logits(T, G, bf16, seed=T + G)
    bias = torch.from_numpy(np.random.default_rng(G).normal(size=G) * 0.1).float() if biased else None
    check(x, bias, k, sigmoid, groups, top_groups, best, renorm, 2.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,best", [(1, 1), (8, 1), (8, 2)])
def test_equal_values_go_to_the_lowest_index(sigmoid, groups, best):
    x = torch.from_numpy(np.random.default_rng(0).integers(-2, 3, size=(200, 64))).float()
    check(x, None, 8, sigmoid, groups, max(1, groups // 2), best)
    check(x, torch.full((64,), 0.25), 8, sigmoid, groups, max(1, groups // 2), best)
    # two biases: values that differ, and many that are equal
    check(x, torch.tensor([0.0, 0.5] * 32), 8, sigmoid, groups, max(1, groups // 2), best)
    check(torch.zeros(3, 64), None, 32, sigmoid, groups, groups, best)


def test_values_nearer_than_a_rounding():
    # c of neighbours 1e-9 apart in 64 bits, in the other order or equal in 32
    G = 64
    x = torch.linspace(-1.0, 1.0, G).repeat(40, 1)
    s = 1.0 / (1.0 + np.exp(-x[0].double().numpy()))
    bias = torch.from_numpy(0.75 - s).float()    # (rounded: all c near 0.75, by 3e-8)
    check(x, bias, 8, True)
    check(x, bias, 8, True, 8, 3, 2)
    check(x, bias, 8, True, 8, 3, 1)
    p = torch.softmax(x[0].double(), 0).numpy()
    check(x, torch.from_numpy(0.1 - p).float(), 8, False)
    check(x, torch.from_numpy(0.1 - p).float(), 8, False, 4, 2, 2)


@pytest.mark.parametrize("G,k,groups,best", [(8, 8, 1, 1), (16, 7, 4, 1), (32, 8, 4, 2), (64, 16, 1, 1), (128, 6, 8, 1),
                                              (256, 8, 8, 2), (500, 32, 1, 1), (1024, 9, 16, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_equal_logits_in_fp32(G, k, groups, best, sigmoid):
    # logits of a bf16 product as fp32: equal ones in most tokens, also at the last choice, and
    # neighbours by one unit in the last place
    x = logits(300, G, True, G).float()
    top = max(1, groups // 2) if k <= G // groups * max(1, groups // 2) else groups
    check(x, None, k, sigmoid, groups, top, best)
    check(x, torch.full((G,), -0.5), k, sigmoid, groups, top, best)
    near = x[:, :1].expand(300, G).contiguous()
    step = torch.from_numpy(np.random.default_rng(G).integers(0, 4, size=(300, G)).astype(np.int32))
    near = (near.view(torch.int32) + step).view(torch.float32)
    check(near, None, k, sigmoid, groups, top, best)


@pytest.mark.parametrize("G,k,groups,top", [(54, 2, 18, 15), (24, 5, 3, 2), (60, 8, 5, 2), (42, 6, 7, 3),
                                            (96, 6, 12, 4), (100, 9, 25, 7), (520, 8, 13, 4)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_in_doubt_of_which_lanes_are_left_over(G, k, groups, top, sigmoid):
    # numbers of groups that do not divide the lanes; many tokens whose groups' sums are
    # equal, or apart by less than they are off by in fp32
    x = torch.round(logits(200, G, False, G) * 2) / 2
    bias = torch.from_numpy(np.random.default_rng(G).integers(0, 3, size=G)).float() / 4
    for b in (None, bias, torch.full((G,), 0.25)):
        check(x, b, k, sigmoid, groups, top, 2)
        check(x.repeat(3, 1) + 1e-6 * logits(600, G, False, 9), b, k, sigmoid, groups, top, 2)
    check(x, bias, k, sigmoid, groups, top, 1)


def test_far_logits():
    x = torch.tensor([[100.0, -100.0, 90.0, 0.0, -90.0, 30.0, -3e38, 3e38]])
    for sigmoid in (False, True):
        check(x, None, 4, sigmoid)
        check(x[:, 1:5], None, 4, sigmoid)
    check(x, torch.tensor([0.0, 5.0, 0.0, 0.0, 9.0, 0.0, 2.0, 0.0]), 4, True)
    # all scores are below 2^-126, each off by TINY: the sum that they are divided by is
    # 1e-20
    check(torch.tensor([[-100.0, -99.0, -98.0]]), None, 2, True, tiny=TINY / 1e-20)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_experts(sigmoid, biased, groups):
    x = logits(40, 64, False, 5)
    x[0] = -np.inf                      # nothing left
    x[1, 3:] = -np.inf                  # fewer than chosen
    x[2, ::2] = float("nan")
    x[3] = float("nan")
    x[4, 7] = np.inf
    x[5, 16:] = -np.inf                 # whole groups
    x[6] = torch.finfo(torch.float32).min   # a mask of the lowest value: available, all equal
    x[7, :60] = torch.finfo(torch.float32).min
    bias = torch.from_numpy(np.random.default_rng(1).normal(size=64)).float() if biased else None
    e, w = run(x, bias, 6, sigmoid, groups, max(1, groups // 2), 2)
    we, ww = M.route(x.double().numpy(), None if bias is None else bias.numpy(), 6, sigmoid, groups,
                     max(1, groups // 2), 2)
    assert np.array_equal(e, we)
    assert np.isfinite(w).all()
    within(w, ww, 64 * U * np.abs(ww) + 1e-30)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,best", [(1, 1), (8, 2), (8, 1)])
def test_biases_that_decide_by_themselves(sigmoid, groups, best):
    x = logits(30, 64, False, 8)
    bias = torch.from_numpy(np.random.default_rng(2).normal(size=64) * 0.1).float()
    bias[5], bias[6], bias[17], bias[40] = float("inf"), -float("inf"), 1e6, -3e7
    bias[41] = float("nan")       # (not available, as with -infinity)
    e, w = run(x, bias, 7, sigmoid, groups, max(1, groups // 2), best)
    b = bias.numpy().copy()
    b[41] = -np.inf
    we, ww = M.route(x.double().numpy(), b, 7, sigmoid, groups, max(1, groups // 2), best)
    assert np.array_equal(e, we)
    within(w, ww, 64 * U * np.abs(ww) + TINY)


@pytest.mark.parametrize("G,k,groups,top_groups", [(384, 16, 8, 3), (1024, 32, 32, 9), (64, 5, 2, 1), (60, 8, 1, 1),
                                                   (16, 4, 4, 2), (8, 3, 1, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_many_values_within_a_rounding(G, k, groups, top_groups, sigmoid):
    # c of every expert within 3e-8 of each other: all of them in doubt in 32 bits
    x = logits(25, G, False, 4)
    for t in range(25):
        s, _ = M.scores(x[t].double().numpy(), sigmoid)
        check(x[t:t + 1], torch.from_numpy(1.0 - s).float(), k, sigmoid, groups, top_groups, 2)
    check(x, torch.from_numpy(1.0 - s).float(), k, sigmoid, groups, top_groups, 2)   # (one token in doubt)
    # neighbouring tokens (which share a warp where there are few experts), one with all of its
    # values in doubt, one with a few, one with none
    y = x.clone()
    y[24] = x[24] + 1e-3 * torch.arange(G)
    y[20] = y[21] = x[24]
    y[21, 3:] = x[21, 3:]
    check(y, torch.from_numpy(1.0 - s).float(), k, sigmoid, groups, top_groups, 2)
    check(y, torch.from_numpy(1.0 - s).float(), k, sigmoid)


def back(x, e, dw, sigmoid, renorm, scale):
    T, G = x.shape
    d = torch.full_like(x, 9.0).cuda()
    fn = dg.route_top_k_backward_bf16 if x.dtype == torch.bfloat16 else dg.route_top_k_backward_fp32
    fn(x.cuda(), torch.from_numpy(e).cuda(), dw.cuda(), d, T, G, e.shape[1], sigmoid, renorm, scale)
    torch.cuda.synchronize()
    return d.cpu().double().numpy()


def check_gradient(x, e, dw, sigmoid, renorm, scale):
    got = back(x, e, dw, sigmoid, renorm, scale)
    xn = x.double().numpy()
    want, mag = M.route_backward(xn, e, dw.numpy(), sigmoid, renorm, scale)
    lim = 2 * (48 + spread(xn)) * U * mag + 1e-30
    if x.dtype == torch.bfloat16:
        lim = lim + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8)
    within(got, want, lim)


@pytest.mark.parametrize("shape", [(1, 8, 2), (33, 256, 8), (9, 60, 6), (130, 1024, 32), (5, 33, 1), (7, 64, 13), (3, 16, 16)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_gradient(shape, sigmoid, renorm, bf16):
    T, G, k = shape
    x = logits(T, G, bf16, seed=G)
    rng = np.random.default_rng(T)
    e = np.stack([rng.permutation(G)[:k] for _ in range(T)]).astype(np.int32)
    check_gradient(x, e, torch.from_numpy(rng.normal(size=(T, k))).float(), sigmoid, renorm, 1.5)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_odd_choices(sigmoid, renorm):
    x = logits(6, 40, False, 2)
    x[1] = -np.inf
    x[2, 5] = float("nan")
    x[3, :30] = 90.0
    e = np.array([[3, 3, 7], [1, 2, 3], [5, 6, 7], [0, 35, -1], [-1, -1, -1], [0, 32, 33]], np.int32)
    dw = torch.from_numpy(np.random.default_rng(0).normal(size=(6, 3))).float()
    dw[4] = float("nan")      # (no choice, no gradient)
    got = back(x, e, dw, sigmoid, renorm, 1.0)
    assert np.isfinite(got).all() and (got[1] == 0).all() and (got[4] == 0).all() and got[2, 5] == 0
    for t in (0, 3, 5):
        check_gradient(x[t:t + 1], e[t:t + 1], dw[t:t + 1], sigmoid, renorm, 1.0)


def test_gradient_reports_an_expert_out_of_range():
    x, dw = logits(2, 16, False, 1), torch.ones(2, 2)
    got = back(x, np.array([[16, 3], [-2, 4]], np.int32), dw, True, False, 1.0)
    assert dg.get_device_status() == 9
    assert np.array_equal(got, back(x, np.array([[-1, 3], [-1, 4]], np.int32), dw, True, False, 1.0))


def test_streams_graphs_and_limits():
    x, bias = logits(300, 256, False, 9).cuda(), torch.randn(256, device="cuda") * 0.1
    e, w = torch.empty(300, 8, dtype=torch.int32, device="cuda"), torch.empty(300, 8, device="cuda")
    d, dw = torch.empty_like(x), torch.randn(300, 8, device="cuda")

    def both(stream=None):
        dg.route_top_k_fp32(x, bias, e, w, 300, 256, 8, True, 8, 4, 2, True, 2.5, stream=stream)
        dg.route_top_k_backward_fp32(x, e, dw, d, 300, 256, 8, True, True, 2.5, stream=stream)

    both()
    torch.cuda.synchronize()
    want = e.clone(), w.clone(), d.clone()
    side = torch.cuda.Stream()
    for t in (e, w, d):
        t.zero_()
    torch.cuda.synchronize()
    both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((e, w, d), want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both()
    for t in (e, w, d):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((e, w, d), want))
    dg.set_num_sms(3)
    try:
        grids = launched(both)
        for t in (e, w, d):
            t.zero_()
        both()
        torch.cuda.synchronize()
    finally:
        dg.set_num_sms(0)
    assert len(grids) == 2 and all(b <= 3 for b, _, _ in grids)
    assert all(torch.equal(a, b) for a, b in zip((e, w, d), want))
