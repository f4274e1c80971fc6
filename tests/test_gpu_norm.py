"""The root-mean-square norm and its gradient on the GPU against their 64-bit
definitions."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import operators_ref as R

pytestmark = pytest.mark.gpu

EPS = 1e-6
# fp32 before the output's rounding: h and two products (3 u), and half the
# error of a sum of squares in chains of at most 32 terms and a tree (below
# 48 u): under 2^-18
REL = 2.0 ** -18


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()


def normal(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def buffers(M, K, ld, ue8m0):
    """Outputs full of what must not stay (codes: NaN) or must (scales past M)."""
    H, Y = (torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Q = torch.full((M, K), 0x7F, dtype=torch.uint8, device="cuda")
    rstd = torch.full((M,), float("nan"), device="cuda")
    if ue8m0:
        return H, Y, Q, torch.full(((K + 511) // 512, ld), 0x55555555, dtype=torch.int32,
                                   device="cuda"), rstd
    return H, Y, Q, torch.full((K // 128, ld), -7.25, device="cuda"), rstd


def forward(X, Rs, W, M, K, ld, ue8m0=False, outs="HYQr", stream=None):
    H, Y, Q, sa, rstd = buffers(M, K, ld, ue8m0)
    fn = dg.rms_norm_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.rms_norm_quantize_fp8_1x128
    fn(X, Rs, W, H if "H" in outs else None, Y if "Y" in outs else None, Q if "Q" in outs else None,
       sa if "Q" in outs else None, rstd if "r" in outs else None, M, K, ld, EPS, stream=stream)
    return H, Y, Q, sa, rstd


def check(X, Rs, W, got, M, K, ue8m0, outs, what):
    H, Y, Q, sa, rstd = got
    h, r, y = R.norm(X, Rs, W, EPS)
    if "H" in outs:
        R.check_close(H, h, R.U32 * h.abs(), f"{what} H")
    if "Y" in outs:
        R.check_close(Y, y, REL * y.abs(), f"{what} Y")
    if "r" in outs:
        assert ((rstd.double() - r).abs() <= REL * r).all(), f"{what} rstd"
    if "Q" in outs:
        kb = K // 128
        s = R.unpack_ue8m0(sa, M, kb) if ue8m0 else R.scales(sa, M, kb).double()
        R.check_scales(s, y, REL, ue8m0, what)
        R.check_codes(Q, s, y, 2 * REL, what)
        if ue8m0:
            assert (sa[:, M:] == 0x55555555).all(), f"{what}: scale columns past M written"
        else:
            assert (sa[:, M:] == -7.25).all(), f"{what}: scale columns past M written"


SHAPES = [(1, 128, 4), (1, 7168, 4), (3, 256, 8), (7, 1536, 8), (33, 640, 36), (130, 2048, 132),
          (5, 8192, 8), (4, 8320, 4), (3, 16384, 4), (700, 384, 700), (1500, 512, 1500),
          (1900, 7168, 1900), (1830, 16384, 1832), (4100, 6272, 4100)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_norm(shape, ue8m0, residual):
    M, K, ld = shape
    X, W = normal(M, K, seed=M + K), normal(K, seed=K, scale=0.5)
    Rs = normal(M, K, seed=K - M, scale=3.0) if residual else None
    outs = "HYQr" if residual else "YQr"
    check(X, Rs, W, forward(X, Rs, W, M, K, ld, ue8m0, outs), M, K, ue8m0, outs, f"{shape}")
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("outs", ["Q", "Y", "Qr", "HQ", "YQ"])
def test_optional_outputs(outs):
    M, K = 19, 896
    X, Rs, W = normal(M, K, seed=1), normal(M, K, seed=2), normal(K, seed=3)
    got = forward(X, Rs, W, M, K, 20, outs=outs)
    check(X, Rs, W, got, M, K, False, outs, outs)
    H, Y, Q, sa, rstd = got
    assert "H" in outs or H.isnan().all()
    assert "Y" in outs or Y.isnan().all()
    assert "r" in outs or rstd.isnan().all()
    assert "Q" in outs or ((Q == 0x7F).all() and (sa == -7.25).all())


def test_extreme_rows():
    """Zero rows, rows below the scale's floor, one dominant value, values near
    the top of bf16 (whose squares pass fp32 are not finite: kept below)."""
    K = 512
    X = normal(6, K, seed=4)
    X[0] = 0
    X[1] *= 1e-20
    X[2, 5] = 3e4
    X[3] *= 1e15
    X[4] = 0
    X[4, 0] = 1e-3
    W = normal(K, seed=5)
    W[:128] = 0                       # a group whose outputs are all zero
    got = forward(X, None, W, 6, K, 8, outs="YQr")
    check(X, None, W, got, 6, K, False, "YQr", "extreme")
    assert (got[2][0] & 0x7F == 0).all() and (got[2][:, :128] & 0x7F == 0).all()


def test_in_place_residual_and_stream():
    """H may be R itself; the call runs on the stream it is given."""
    M, K = 40, 1024
    X, Rs, W = normal(M, K, seed=6), normal(M, K, seed=7), normal(K, seed=8)
    h = X.double() + Rs.double()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y = torch.empty_like(X)
    with torch.cuda.stream(s):
        big = torch.ones(64 << 20, device="cuda")
        for _ in range(20):
            big.mul_(1.0)
        late = X * 1.0
        dg.rms_norm_quantize_fp8_1x128(late, Rs, W, Rs, Y, None, None, None, M, K, 0, EPS, stream=s)
    s.synchronize()
    R.check_close(Rs, h, R.U32 * h.abs(), "H in place")


def test_graph_capture_follows_new_inputs():
    M, K = 17, 2048
    X, W = normal(M, K, seed=9), normal(K, seed=10)
    Q = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(K // 128, 20, device="cuda")
    call = lambda: dg.rms_norm_quantize_fp8_1x128(X, None, W, None, None, Q, sa, None, M, K, 20, EPS)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    X.copy_(normal(M, K, seed=11))
    g.replay()
    torch.cuda.synchronize()
    y = R.norm(X, None, W, EPS)[2]
    s = R.scales(sa, M, K // 128).double()
    R.check_scales(s, y, REL, False, "graph")
    R.check_codes(Q, s, y, 2 * REL, "graph")


def backward(dY, H, rstd, W, dR, dX=None, sms=0):
    M, K = H.shape
    n = dg.rms_norm_backward_workspace_bytes(M, K)
    # the workspace's contents are not read before they are written
    work = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    dX = torch.full((M, K), float("nan"), dtype=torch.bfloat16, device="cuda") if dX is None else dX
    dW = torch.full((K,), float("nan"), device="cuda")
    dg.rms_norm_backward(dY, H, rstd, W, dR, dX, dW, work, n, M, K)
    return dX, dW


def check_backward(dY, H, rstd, W, dR, dX, dW, what):
    M = H.shape[0]
    dx, dw = R.norm_backward(dY, H, rstd, W, dR)
    xh = H.double() * rstd.double()[:, None]
    g = dY.double() * W.double()
    mag = rstd.double()[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    R.check_close(dX, dx, REL * (mag + (dR.double().abs() if dR is not None else 0.0)), f"{what} dX")
    # a block's chain of rows, then at most 304 partial sums in 8 chains
    lim = (64 + M / 16) * 2 * R.U32 * (dY.double() * xh).abs().sum(0)
    bad = ~((dW.double() - dw).abs() <= lim)
    assert not bad.any(), f"{what} dW: {int(bad.sum())} off"


@pytest.mark.parametrize("shape", [(1, 128), (1, 7168), (2, 256), (33, 640), (150, 2048), (305, 1024),
                                   (611, 384), (9, 8320), (4, 16384), (2500, 512),
                                   (460, 7168), (500, 16384), (1300, 2048)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient(shape, residual):
    M, K = shape
    H, W = normal(M, K, seed=M, scale=2.0), normal(K, seed=K, scale=0.5)
    dY = normal(M, K, seed=M + 1, scale=0.03)
    dR = normal(M, K, seed=M + 2, scale=0.03) if residual else None
    rstd = torch.rsqrt(H.float().square().mean(-1) + EPS)
    dX, dW = backward(dY, H, rstd, W, dR)
    check_backward(dY, H, rstd, W, dR, dX, dW, f"{shape}")
    again = backward(dY, H, rstd, W, dR)
    assert torch.equal(again[0], dX) and torch.equal(again[1], dW), "same inputs, other bits"


def test_norm_gradient_in_place_and_few_sms():
    """dX may be dR; a limit on the SMs changes the split, not the result's bounds."""
    M, K = 100, 1024
    H, W, dY, dR = (normal(M, K, seed=20), normal(K, seed=21), normal(M, K, seed=22),
                    normal(M, K, seed=23))
    rstd = torch.rsqrt(H.float().square().mean(-1) + EPS)
    keep = dR.clone()
    dg.set_num_sms(3)
    try:
        dX, dW = backward(dY, H, rstd, W, dR, dX=dR)
    finally:
        dg.set_num_sms(0)
    assert dX.data_ptr() == dR.data_ptr()
    check_backward(dY, H, rstd, W, keep, dX, dW, "in place")


@pytest.mark.parametrize("shape,sms", [((1000, 4224), 0), ((930, 6400), 0), ((950, 8192), 0),
                                       ((100, 5120), 3), ((31, 8064), 1), ((20, 16384), 3),
                                       ((23, 12416), 1)],
                         ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else f"{s}sms")
@pytest.mark.parametrize("residual", [False, True])
def test_norm_gradient_of_long_rows(shape, sms, residual):
    """Rows that take two vectors a thread, many rows per block (every slot of
    the ring several times), dX in place of dR."""
    M, K = shape
    H, W = normal(M, K, seed=M, scale=2.0), normal(K, seed=K, scale=0.5)
    dY = normal(M, K, seed=M + 1, scale=0.03)
    dR = normal(M, K, seed=M + 2, scale=0.03) if residual else None
    rstd = torch.rsqrt(H.float().square().mean(-1) + EPS)
    keep = dR.clone() if residual else None
    dg.set_num_sms(sms)
    try:
        dX, dW = backward(dY, H, rstd, W, dR, dX=dR)
    finally:
        dg.set_num_sms(0)
    check_backward(dY, H, rstd, W, keep, dX, dW, f"{shape}")


def test_norm_gradient_of_no_rows():
    dW = torch.full((256,), float("nan"), device="cuda")
    dg.rms_norm_backward(None, None, None, None, None, None, dW, None, 0, 0, 256)
    assert (dW == 0).all()


def test_forward_then_gradient_matches_autograd():
    """The pair of calls against autograd of the definition in 64 bits."""
    M, K = 12, 768
    X, Rs, W, dY = (normal(M, K, seed=30), normal(M, K, seed=31), normal(K, seed=32),
                    normal(M, K, seed=33))
    H, _, _, _, rstd = forward(X, Rs, W, M, K, 12, outs="HYr")
    dX, dW = backward(dY, H, rstd, W, None)
    h, w = H.double().requires_grad_(), W.double().requires_grad_()
    (h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w * dY.double()).sum().backward()
    # rstd is that of the sum before its rounding to bf16: off by up to 2^-8
    # of itself, and dX with it
    assert (dX.double() - h.grad).norm() <= 2 * R.BF16_ROUND * h.grad.norm()
    assert (dW.double() - w.grad).norm() <= 2 * R.BF16_ROUND * w.grad.norm()


def test_rows_past_32_bit_offsets():
    """More than 2^31 elements: the last rows are addressed in 64 bits."""
    K = 16384
    M = (1 << 31) // K + 3
    X = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    X[-4:] = normal(4, K, seed=40)
    W = normal(K, seed=41)
    ld = (M + 3) // 4 * 4
    Q = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(K // 128, ld, device="cuda")
    dg.rms_norm_quantize_fp8_1x128(X, None, W, None, None, Q, sa, None, M, K, ld, EPS)
    y = R.norm(X[-4:], None, W, EPS)[2]
    s = sa[:, M - 4:M].t().double()
    R.check_scales(s, y, REL, False, "tail")
    R.check_codes(Q[-4:], s, y, 2 * REL, "tail")
    assert (Q[:M - 4] & 0x7F == 0).all()   # (zeros of either sign)
