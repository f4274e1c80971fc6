"""A limit on the SMs bounds what the operators around the GEMMs launch: every
grid of at most as many blocks as SMs, results as without it."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import operators_ref as R
from tests import test_gpu_bf16_ragged as P
from tests import test_gpu_norm as N
from tests.launches import launched
from tests.test_gpu_bf16_ragged import ints
from tests.test_gpu_swiglu import normal
from tests.test_gpu_swiglu_ring import Activation

pytestmark = pytest.mark.gpu

LIMITS = [1, 3, 16, 132]


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    dg.set_num_sms(0)


def within(sms, call):
    """The call under the limit, and its grids checked."""
    dg.set_num_sms(sms)
    try:
        call(None)
        grids = launched(call)
    finally:
        dg.set_num_sms(0)
    assert grids and all(blocks <= sms for blocks, _, _ in grids), (sms, grids)


# few tiles and deep reductions (which otherwise split), many groups of few rows,
# a few rows in all
PRODUCTS = [("nt", [38, 36, 40, 37], 3832, 8048), ("nt", [5] * 12, 520, 8192), ("nn", [33], 128, 6000),
            ("nn", [14] * 27, 1032, 2056), ("tn", [3000, 0, 20], 64, 128), ("tn", [5001, 7], 256, 264),
            ("nt", [1], 7168, 2048), ("nn", [2, 0, 1], 2048, 1024), ("tn", [3, 1], 520, 328),
            ("nt", [300, 0, 41, 513], 520, 456)]


@pytest.mark.parametrize("form,sizes,N_,K", PRODUCTS)
@pytest.mark.parametrize("sms", LIMITS)
def test_products(form, sizes, N_, K, sms):
    A, B = P.inputs(form, sizes, N_, K, seed=sms)
    n, T, G = ints(sizes), A.shape[0], len(sizes)
    D = torch.full((G, K, N_) if form == "tn" else (T, N_), P.KEEP, dtype=torch.bfloat16, device="cuda")
    if form == "tn":
        call = lambda s: dg.k_grouped_gemm_bf16_tn_ragged(A, B, D, n, G, K, N_, T, stream=s)
    else:
        fn = dg.m_grouped_gemm_bf16_nt_ragged if form == "nt" else dg.m_grouped_gemm_bf16_nn_ragged
        call = lambda s: fn(A, B, D, n, T, N_, K, G, stream=s)
    within(sms, call)
    P.check(form, A, B, sizes, D, f"{form} on {sms} SMs")


def test_forced_tilings_past_the_limit_are_refused():
    sizes = [40] * 12
    A, B = P.inputs("nt", sizes, 512, 1024, seed=1)
    dg.set_num_sms(8)
    try:
        dg.debug_force_ragged_plan(False, 128, 64, 4)
        with pytest.raises(dg.DGError) as e:
            P.run("nt", A, B, sizes, 512)
        assert e.value.status == 2
        dg.debug_force_ragged_plan(False, 128, 64, 1)
        D = P.run("nt", A, B, sizes, 512)
    finally:
        dg.debug_force_ragged_plan()
        dg.set_num_sms(0)
    P.check("nt", A, B, sizes, D, "forced")


@pytest.mark.parametrize("shape", [(1, 7168), (7, 1536), (200, 128), (150, 384), (700, 2048), (40, 8320),
                                   (300, 6144), (1500, 512), (45, 16384), (400, 7168)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("sms", LIMITS)
def test_norm(shape, ue8m0, sms):
    M, K = shape
    ld = (M + 3) // 4 * 4
    X, Rs, W = normal(M, K, seed=M), normal(M, K, seed=K, scale=3.0), normal(K, seed=sms)
    H, Y, Q, sa, rstd = got = N.buffers(M, K, ld, ue8m0)
    fn = dg.rms_norm_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.rms_norm_quantize_fp8_1x128
    within(sms, lambda s: fn(X, Rs, W, H, Y, Q, sa, rstd, M, K, ld, N.EPS, stream=s))
    N.check(X, Rs, W, got, M, K, ue8m0, "HYQr", f"{shape} on {sms} SMs")
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("shape", [(0, 256), (1, 7168), (2, 256), (33, 640), (150, 2048), (305, 1024),
                                   (611, 384), (9, 8320), (45, 16384), (2500, 512), (200, 128),
                                   (460, 7168), (300, 5120)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("sms", LIMITS)
def test_norm_gradient(shape, residual, sms):
    M, K = shape
    H, W = normal(M, K, seed=M, scale=2.0), normal(K, seed=K, scale=0.5)
    dY = normal(M, K, seed=M + 1, scale=0.03)
    dR = normal(M, K, seed=M + 2, scale=0.03) if residual else None
    rstd = torch.rsqrt(H.float().square().mean(-1) + N.EPS)
    n = dg.rms_norm_backward_workspace_bytes(M, K)
    work = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    dX = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    dW = torch.full((K,), float("nan"), device="cuda")
    within(sms, lambda s: dg.rms_norm_backward(dY, H, rstd, W, dR, dX, dW, work, n, M, K, stream=s))
    if M == 0:
        assert (dW == 0).all()
        return
    # (as N.check_backward, whose bound for dW supposes the rows to be spread over
    # the blocks: here one block may add up a chain of M / sms rows)
    dx, dw = R.norm_backward(dY, H, rstd, W, dR)
    xh, g = H.double() * rstd.double()[:, None], dY.double() * W.double()
    mag = rstd.double()[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    R.check_close(dX, dx, N.REL * (mag + (dR.double().abs() if residual else 0.0)), "dX")
    lim = (64 + M / min(sms, 16)) * 2 * R.U32 * (dY.double() * xh).abs().sum(0)
    assert ((dW.double() - dw).abs() <= lim).all(), "dW"
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("shape", [(1, 1, 128), (1, 37, 256), (1, 200, 2048), (1, 4111, 640), (3, 57, 384),
                                   (2, 301, 4224), (1, 60, 16384)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ue8m0,outs", [(False, "YQC"), (True, "Q")])
@pytest.mark.parametrize("sms", LIMITS)
def test_activation(shape, ue8m0, outs, sms):
    a = Activation(*shape, ue8m0, outs, seed=sum(shape))
    within(sms, a)
    a.check()


MASKED = [(3, 64, 512, [64, 0, 33]), (8, 650, 384, [650, 3, 0, 0, 129, 640, 32, 1]), (2, 40, 256, [0, 0])]


@pytest.mark.parametrize("G,M,I,rows", MASKED)
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("sms", LIMITS)
def test_masked_activation(G, M, I, rows, ue8m0, sms):
    from tests.test_gpu_swiglu import check
    a = Activation(G, M, I, ue8m0, "YQC", seed=M)
    for z, n in enumerate(rows):
        a.GU[z, n:] = float("nan")
    mm = ints(rows)
    fn = dg.swiglu_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.swiglu_quantize_fp8_1x128
    within(sms, lambda s: fn(a.GU, a.Y, a.Q, a.sa, a.CQ, a.csa, G, M, I, a.ld, masked_m=mm, stream=s))
    check(a.GU, (a.Y, a.Q, a.sa, a.CQ, a.csa), rows, ue8m0, f"masked on {sms} SMs")
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("G,M,I,rows", MASKED + [(1, 700, 2048, None)])
@pytest.mark.parametrize("sms", LIMITS)
def test_activation_gradient(G, M, I, rows, sms):
    """The same bits as without a limit."""
    GU, dY = normal(G, M, 2 * I, seed=M, scale=1.5), normal(G, M, I, seed=I, scale=0.05)
    ld = (M + 3) // 4 * 4
    CQ = torch.zeros(G, M, 2 * I, dtype=torch.uint8, device="cuda")
    csa = torch.zeros(G, 2 * I // 128, ld, device="cuda")
    dg.quantize_fp8_1x128(GU, CQ, csa, G, M, 2 * I, ld)
    mm = None if rows is None else ints(rows)
    outs = [[torch.full((G, M, w * I), -3.0, dtype=torch.bfloat16, device="cuda") for w in (2, 1)]
            for _ in range(2)]
    call = lambda o, s: dg.swiglu_backward_fp8_1x128(CQ, csa, dY, o[0], o[1], G, M, I, ld, masked_m=mm,
                                                     stream=s)
    call(outs[0], None)
    within(sms, lambda s: call(outs[1], s))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert dg.get_device_status() == 0
