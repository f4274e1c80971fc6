"""Refusals of routing, the experts' rows, dispatch and combine: arguments are
checked on the host before a device is touched (no GPU needed)."""
import pytest

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests.test_operators_abi import INVALID, MISALIGNED, OK, SHAPE, P, status


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


ROUTE = dict(logits=P, bias=P, experts=P, weights=P, T=5, num_experts=64, top_k=6, sigmoid=True,
             num_groups=8, top_groups=4, group_best=2, renormalize=True, scale=1.0)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(weights=None), INVALID),
    (dict(T=-1), INVALID), (dict(num_experts=0), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=33, top_groups=8), SHAPE), (dict(num_experts=1025, num_groups=1, top_groups=1), SHAPE),
    (dict(num_groups=7), INVALID), (dict(num_groups=0), INVALID), (dict(top_groups=0), INVALID),
    (dict(top_groups=9), INVALID), (dict(group_best=3), INVALID), (dict(group_best=0), INVALID),
    (dict(top_groups=1, top_k=9), INVALID), (dict(num_groups=64, top_groups=64), SHAPE),
    (dict(T=1 << 28), SHAPE), (dict(bias=P + 2), MISALIGNED), (dict(experts=P + 2), MISALIGNED),
    (dict(weights=P + 1), MISALIGNED), (dict(logits=P + 1), MISALIGNED),
    (dict(T=0), OK), (dict(T=0, logits=None, experts=None, weights=None), OK)])
@pytest.mark.parametrize("fn", ["route_top_k_fp32", "route_top_k_bf16"])
def test_route_refusals(fn, kw, code):
    assert status(getattr(dg, fn), {**ROUTE, **kw}) == code


def test_route_alignment_is_that_of_the_logits():
    assert status(dg.route_top_k_fp32, {**ROUTE, "logits": P + 2}) == MISALIGNED
    assert status(dg.route_top_k_bf16, {**ROUTE, "logits": P + 1}) == MISALIGNED


ROUTE_BWD = dict(logits=P, experts=P, d_weights=P, d_logits=P, T=5, num_experts=64, top_k=6)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), INVALID), (dict(experts=None), INVALID), (dict(d_weights=None), INVALID),
    (dict(d_logits=None), INVALID), (dict(T=-1), INVALID), (dict(top_k=33), SHAPE),
    (dict(num_experts=2000), SHAPE), (dict(d_logits=P + 1), MISALIGNED), (dict(d_weights=P + 2), MISALIGNED),
    (dict(T=0), OK)])
@pytest.mark.parametrize("fn", ["route_top_k_backward_fp32", "route_top_k_backward_bf16"])
def test_route_gradient_refusals(fn, kw, code):
    assert status(getattr(dg, fn), {**ROUTE_BWD, **kw}) == code


ROWS = dict(experts=P, rows=P, T=5, top_k=2, num_groups=4)
COMMON = [(dict(experts=None), INVALID), (dict(rows=None), INVALID), (dict(T=-1), INVALID),
          (dict(top_k=0), INVALID), (dict(num_groups=0), INVALID), (dict(num_groups=1025), SHAPE),
          (dict(top_k=33), SHAPE), (dict(T=1 << 30), SHAPE), (dict(experts=P + 2), MISALIGNED),
          (dict(rows=P + 2), MISALIGNED)]


@pytest.mark.parametrize("kw,code", COMMON + [(dict(ms=None), INVALID), (dict(ms=P + 1), MISALIGNED)])
def test_ragged_rows_refusals(kw, code):
    assert status(dg.expert_rows_ragged, {**ROWS, "ms": P, **kw}) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(ms=None), INVALID), (dict(m_indices=None), INVALID), (dict(M_total=-128), INVALID),
    (dict(M_total=100), SHAPE), (dict(m_indices=P + 2), MISALIGNED)])
def test_contiguous_rows_refusals(kw, code):
    assert status(dg.expert_rows_contiguous, {**ROWS, "ms": P, "m_indices": P, "M_total": 512, **kw}) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(masked_m=None), INVALID), (dict(max_m=-1), INVALID), (dict(max_m=1 << 29), SHAPE)])
def test_masked_rows_refusals(kw, code):
    assert status(dg.expert_rows_masked, {**ROWS, "masked_m": P, "max_m": 64, **kw}) == code


MOVE = dict(X=P, rows=P, D=P, T=5, K=256, top_k=2, num_rows=10)


@pytest.mark.parametrize("kw,code", [
    (dict(X=None), INVALID), (dict(rows=None), INVALID), (dict(D=None), INVALID), (dict(T=-1), INVALID),
    (dict(num_rows=-1), INVALID), (dict(K=0), SHAPE), (dict(K=12), SHAPE), (dict(top_k=40), SHAPE),
    (dict(X=P + 8), MISALIGNED), (dict(D=P + 4), MISALIGNED), (dict(rows=P + 2), MISALIGNED), (dict(T=0), OK)])
def test_dispatch_refusals(kw, code):
    assert status(dg.dispatch_rows_bf16, {**MOVE, **kw}) == code


MOVE8 = dict(Q=P, rows=P, A=P, ld_out=64, T=5, K=256, top_k=2, num_groups=4, max_m=64)


@pytest.mark.parametrize("kw,code", [
    (dict(Q=None), INVALID), (dict(rows=None), INVALID), (dict(A=None), INVALID), (dict(s=None), INVALID),
    (dict(o=None), INVALID), (dict(ld=4), INVALID), (dict(ld=10), MISALIGNED), (dict(ld_out=60), INVALID),
    (dict(ld_out=65), MISALIGNED), (dict(num_groups=0), INVALID), (dict(max_m=-1), INVALID),
    (dict(K=64), SHAPE), (dict(K=200), SHAPE), (dict(max_m=1 << 30, ld_out=1 << 30), SHAPE),
    (dict(s=P + 4), MISALIGNED), (dict(o=P + 8), MISALIGNED), (dict(A=P + 8), MISALIGNED), (dict(T=0), OK)])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_dispatch_fp8_refusals(ue8m0, kw, code):
    fn = dg.dispatch_rows_fp8_1x128_ue8m0 if ue8m0 else dg.dispatch_rows_fp8_1x128
    names = dict(s="sfa", o="sfa_out", ld="ld_sfa") if ue8m0 else dict(s="sa", o="sa_out", ld="ld_sa")
    a = {**MOVE8, "s": P, "o": P, "ld": 8, **kw}
    assert status(fn, {names.get(k, k): v for k, v in a.items()}) == code


SUM = dict(Y=P, rows=P, weights=P, R=P, out=P, T=5, K=256, top_k=2, num_rows=10)


@pytest.mark.parametrize("kw,code", [
    (dict(Y=None), INVALID), (dict(rows=None), INVALID), (dict(out=None), INVALID), (dict(T=-1), INVALID),
    (dict(num_rows=-1), INVALID), (dict(K=4), SHAPE), (dict(K=260), SHAPE), (dict(top_k=33), SHAPE),
    (dict(R=P + 8), MISALIGNED), (dict(weights=P + 2), MISALIGNED), (dict(out=P + 2), MISALIGNED),
    (dict(T=0), OK)])
def test_combine_refusals(kw, code):
    assert status(dg.combine_rows, {**SUM, **kw}) == code


SUM_BWD = dict(dO=P, Y=P, rows=P, weights=P, dY=P, d_weights=P, T=5, K=256, top_k=2, num_rows=10)


@pytest.mark.parametrize("kw,code", [
    (dict(dO=None), INVALID), (dict(Y=None), INVALID), (dict(rows=None), INVALID), (dict(dY=None), INVALID),
    (dict(T=-1), INVALID), (dict(K=20), SHAPE), (dict(top_k=0), INVALID), (dict(dO=P + 8), MISALIGNED),
    (dict(dY=P + 8), MISALIGNED), (dict(d_weights=P + 2), MISALIGNED), (dict(T=0), OK)])
def test_combine_gradient_refusals(kw, code):
    assert status(dg.combine_rows_backward, {**SUM_BWD, **kw}) == code


LOSS = dict(X=P, W=P, targets=P, loss=P, lse=P, workspace=P, workspace_bytes=1 << 40, T=5, V=1000, K=256)
LOSS_COMMON = [(dict(X=None), INVALID), (dict(W=None), INVALID), (dict(targets=None), INVALID),
               (dict(workspace=None), INVALID), (dict(workspace_bytes=64), INVALID), (dict(T=-1), INVALID),
               (dict(V=0), INVALID), (dict(K=0), INVALID), (dict(K=12), SHAPE), (dict(V=2 ** 31 - 1), SHAPE),
               (dict(T=1 << 23), SHAPE), (dict(V=1 << 27, K=128), SHAPE), (dict(T=1 << 20, V=1 << 20), SHAPE),
               (dict(X=P + 8), MISALIGNED), (dict(W=P + 2), MISALIGNED), (dict(workspace=P + 4), MISALIGNED),
               (dict(targets=P + 2), MISALIGNED), (dict(lse=P + 2), MISALIGNED)]


@pytest.mark.parametrize("V,code", [(1 << 29, SHAPE), ((1 << 29) - 1, INVALID)])
def test_the_largest_vocabulary(V, code):
    # (within the limit it is the workspace that is refused, before anything else)
    assert status(dg.linear_cross_entropy, {**LOSS, "V": V, "K": 8, "workspace_bytes": 64}) == code


@pytest.mark.parametrize("kw,code", LOSS_COMMON + [
    (dict(loss=None, lse=None), INVALID), (dict(loss=P + 1), MISALIGNED),
    (dict(T=0, X=None, W=None, targets=None, loss=None, lse=None, workspace=None), OK)])
def test_loss_refusals(kw, code):
    assert status(dg.linear_cross_entropy, {**LOSS, **kw}) == code


LOSS_BWD = dict(X=P, W=P, targets=P, lse=P, d_loss=P, dX=P, dW=P, workspace=P, workspace_bytes=1 << 40, T=5,
                V=1000, K=256)


@pytest.mark.parametrize("kw,code", LOSS_COMMON + [
    (dict(lse=None), INVALID), (dict(d_loss=None), INVALID), (dict(dX=None, dW=None), INVALID),
    (dict(dX=P + 8), MISALIGNED), (dict(dW=P + 8), MISALIGNED), (dict(d_loss=P + 2), MISALIGNED),
    (dict(T=0, dW=None), OK)])
def test_loss_gradient_refusals(kw, code):
    assert status(dg.linear_cross_entropy_backward, {**LOSS_BWD, **kw}) == code


def test_loss_workspaces():
    f, b = dg.linear_cross_entropy_workspace_bytes, dg.linear_cross_entropy_backward_workspace_bytes
    for n in (f, b):
        assert n(0, 0, 0) == 0 and n(5, 0, 8) >= 0 and n(5, 7, 0) >= 0
        assert n(0, 1000, 256) == 0 and n(-1, 5, 8) == -1 and n(5, -1, 8) == -1 and n(5, 5, -1) == -1
    for T, V in ((1, 1), (1, 131072), (4096, 131072), (100000, 50003)):
        K = 2048
        # far below the logits', where there are many
        assert f(T, V, K) <= T * (V / (2 if T <= 64 else 4) + 300) and f(T, V, K) >= 8 * T
        words = b(T, V, K) // (2 * T)
        # a piece of the gradient of the logits; dX in fp32, of a few tokens in parts
        assert b(T, V, K) <= max(2 * T * 4352, 400 << 20) + max(4 * T * K, 64 << 20) + 1024
        assert words >= min(V, 4096)
