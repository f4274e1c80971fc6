"""Outputs that pass fp32 before they are quantised to 8 bits: finite bf16
inputs whose product is above the largest fp32 number.  The group's maximum
counts as that number, so its scale is finite, such an element gets the largest
code of its sign, and the others keep theirs."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import operators_ref as R

pytestmark = pytest.mark.gpu

TOP = float(torch.finfo(torch.float32).max)


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()


def check(Q, scale, y):
    """Q [K], scale [K/128] of the 64-bit y [K]."""
    past = y.abs() > TOP
    assert past.any() and (Q[past] == torch.where(y[past] > 0, 0x7E, 0xFE)).all()
    a = R.group_amax(y).clamp_max(TOP)
    assert torch.isfinite(scale).all()
    # (two rounded factors before the product, one quotient: 2^-20 is ample; a
    # power of two not below it)
    assert (scale >= a / 448 * (1 - 2.0 ** -20)).all() and (scale <= a / 224).all()
    kept = ~past
    R.check_codes((Q * kept)[None], scale[None], (y * kept)[None], 2.0 ** -18, "codes")


@pytest.mark.parametrize("ue8m0", [False, True])
def test_activation(ue8m0):
    I, M = 256, 3
    GU = torch.ones(1, M, 2 * I, dtype=torch.bfloat16, device="cuda")
    GU[0, 0, 5], GU[0, 0, I + 5] = 1e30, 1e30            # + inf in fp32
    GU[0, 1, 200], GU[0, 1, I + 200] = 2e38, -3e38       # - inf, in the second group
    GU[0, 1, 201], GU[0, 1, I + 201] = 1e19, 1e19        # 1e38: keeps its code
    GU[0, 2, 7], GU[0, 2, I + 7] = -3e38, 1e30           # (a gate that far below: zero)
    GU[0, 2, 9], GU[0, 2, I + 9] = 3e38, 1e30
    GU[0, 2, 8], GU[0, 2, I + 8] = 1e19, 3e19            # near the top, finite
    Y = torch.zeros(1, M, I, dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros(1, M, I, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(1, 1 if ue8m0 else I // 128, 4, dtype=torch.int32 if ue8m0 else torch.float32,
                     device="cuda")
    CQ, csa = torch.zeros(1, M, 2 * I, dtype=torch.uint8, device="cuda"), torch.zeros(1, 4, 4, device="cuda")
    fn = dg.swiglu_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.swiglu_quantize_fp8_1x128
    fn(GU, Y, Q, sa, CQ, csa, 1, M, I, 4)
    s = (R.unpack_ue8m0(sa[0], M, 2) if ue8m0 else R.scales(sa[0], M, 2).double())
    for m in range(M):
        check(Q[0, m], s[m], R.swiglu(GU[0])[m])
    assert Q[0, 0, 5] == 0x7E and Q[0, 1, 200] == 0xFE
    assert torch.isposinf(Y[0, 0, 5]) and torch.isneginf(Y[0, 1, 200])
    want, wants = torch.zeros_like(CQ), torch.zeros_like(csa)
    dg.quantize_fp8_1x128(GU, want, wants, 1, M, 2 * I, 4)
    assert torch.equal(CQ, want) and torch.equal(csa, wants)


@pytest.mark.parametrize("K", [256, 8320])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_norm(K, ue8m0):
    X = torch.zeros(2, K, dtype=torch.bfloat16, device="cuda")
    X[0, 3], X[1, 130] = 100.0, -100.0                   # alone in their rows: y = +- sqrt(K)
    X[0, 4], X[1, 131] = 1e-3, 1e-3
    W = torch.full((K,), 3e38, dtype=torch.bfloat16, device="cuda")
    Q = torch.zeros(2, K, dtype=torch.uint8, device="cuda")
    sa = torch.zeros((K + 511) // 512 if ue8m0 else K // 128, 4,
                     dtype=torch.int32 if ue8m0 else torch.float32, device="cuda")
    fn = dg.rms_norm_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.rms_norm_quantize_fp8_1x128
    fn(X, None, W, None, None, Q, sa, None, 2, K, 4, 1e-6)
    y = R.norm(X, None, W, 1e-6)[2]
    s = R.unpack_ue8m0(sa, 2, K // 128) if ue8m0 else R.scales(sa, 2, K // 128).double()
    for m in range(2):
        check(Q[m], s[m], y[m])
    assert Q[0, 3] == 0x7E and Q[1, 130] == 0xFE
