"""The choice of experts where fp32 does not decide it: scores below what fp32 holds,
biases that cancel in a group's sum, and infinite ones beside others.  The choice is
exact, the weights' bounds are those of test_gpu_route.py."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import moe_ref as M
from tests.test_gpu_route import TINY, U, check, logits, run, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    assert dg.get_device_status() == 0


def test_groups_of_scores_below_normal_numbers():
    # softmax scores of e^-86.25 are held, those of e^-87.5 are below 2^-126: the second
    # group's sum is the larger one by less than the third's single score
    x = torch.tensor([[0.0, -200.0, -86.4, -87.5, -86.25, -200.0]])
    check(x, None, 2, False, 3, 2, 2)
    check(x.repeat(70, 1) - torch.arange(70)[:, None], None, 2, False, 3, 2, 2)
    # in a row of 256, among others
    y = torch.full((3, 256), -300.0)
    y[:, 0], y[:, 32:34], y[:, 64:66] = 0.0, x[0, 2:4], x[0, 4:6]
    check(y, None, 9, False, 8, 2, 2)
    check(y.to(torch.bfloat16), None, 9, False, 8, 2, 2)


@pytest.mark.parametrize("unit", [0.0, 1e-40, 3e-37, 1e-30])
def test_biases_next_to_scores_below_normal_numbers(unit):
    # one score has it all, the others are 1e-34 to 1e-56; biases as small, not all equal, or
    # zero but for one that is not available
    for G, k in ((16, 5), (64, 8), (256, 8)):
        x = logits(40, G, False, G, scale=4.0) - 100.0
        x[:, 3] = 0.0
        bias = torch.from_numpy(np.random.default_rng(G).normal(size=G) * unit).float()
        bias[5] = float("nan")
        b = bias.numpy().copy()
        b[5] = -np.inf
        for groups, top in ((1, 1), (4, 3)):
            e, w = run(x, bias, k, False, groups, top, 2)
            we, ww = M.route(x.double().numpy(), b, k, False, groups, top, 2)
            assert np.array_equal(e, we), np.argwhere(e != we)[:5].tolist()
            within(w, ww, (48 + 130) * U * np.abs(ww) + TINY)


@pytest.mark.parametrize("G,groups,top,k", [(64, 8, 3, 8), (256, 8, 4, 8), (16, 8, 3, 4), (60, 5, 2, 6), (512, 16, 5, 9)])
@pytest.mark.parametrize("size", [2.0, 100.0, 3000.0])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_biases_that_cancel_in_a_groups_sum(G, groups, top, k, size, sigmoid):
    # a group's two largest c are near +size and -size: each is rounded by what `size` is, their
    # sum is of the size of the scores
    per = G // groups
    bias = torch.full((groups, per), -2.0)
    bias[:, 0], bias[:, per - 1] = 1.0, -1.0
    x = logits(400, G, False, G)
    check(x, size * bias.flatten(), k, sigmoid, groups, top, 2)
    check(x.to(torch.bfloat16), size * bias.flatten(), k, sigmoid, groups, top, 2)


@pytest.mark.parametrize("G,k,groups,top", [(64, 6, 1, 1), (256, 8, 1, 1), (256, 8, 8, 4), (16, 4, 1, 1), (512, 32, 8, 3)])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_an_infinite_bias_beside_large_ones(G, k, groups, top, sigmoid, sign):
    # c of the others near 1000, many of them within a rounding of that; and of a few units
    x = logits(200, G, False, G)
    small = torch.from_numpy(np.random.default_rng(G).normal(size=G)).float()
    for bias in (1000.0 + 1e-3 * small, small):
        bias[G // 2] = sign * float("inf")
        check(x, bias, k, sigmoid, groups, top, 2)
        check(x, bias, k, sigmoid, groups, top, 1)


@pytest.mark.parametrize("G,k", [(64, 3), (256, 8), (16, 4), (1024, 32)])
@pytest.mark.parametrize("groups,best", [(1, 1), (4, 1), (4, 2)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_more_infinite_biases_than_choices(G, k, groups, best, sigmoid):
    # all of them equal: the lowest indices, whichever lanes hold them
    x = logits(50, G, False, G)
    at = np.random.default_rng(k).permutation(G)[:min(G, 2 * k + 3)]
    bias = torch.from_numpy(np.random.default_rng(G).normal(size=G)).float()
    bias[torch.from_numpy(at)] = float("inf")
    check(x, bias, k, sigmoid, groups, max(1, groups // 2), best)
    few = torch.zeros(G)
    few[torch.from_numpy(at[:max(1, k - 1)])] = float("inf")   # (and one more by its score)
    few[at[-1]] = -1.0
    check(x, few, k, sigmoid, groups, max(1, groups // 2), best)
