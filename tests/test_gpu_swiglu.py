"""The gated activation, its 8-bit checkpoint and its gradient on the GPU
against their 64-bit definitions."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import operators_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()


def rel(g):
    """Relative error of silu(g) u in fp32: the hardware exponential is off by
    2 + 1.173 |g| ulp at most, the quotient by 2 ulp and the products by one.
    (Rows without a token may hold NaN.)"""
    return (8 + 1.173 * float(g.abs().nan_to_num(0.0).max())) * 2 * R.U32


def normal(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def forward(GU, ld, masked=None, ue8m0=False, outs="YQC"):
    G, M, I2 = GU.shape
    I = I2 // 2
    Y = torch.full((G, M, I), -3.0, dtype=torch.bfloat16, device="cuda")
    Q = torch.full((G, M, I), 0x7F, dtype=torch.uint8, device="cuda")
    sa = (torch.full((G, (I + 511) // 512, ld), 0x55555555, dtype=torch.int32, device="cuda") if ue8m0
          else torch.full((G, I // 128, ld), -7.25, device="cuda"))
    CQ = torch.full((G, M, I2), 0x7F, dtype=torch.uint8, device="cuda")
    csa = torch.full((G, I2 // 128, ld), -7.25, device="cuda")
    fn = dg.swiglu_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.swiglu_quantize_fp8_1x128
    fn(GU, Y if "Y" in outs else None, Q if "Q" in outs else None, sa if "Q" in outs else None,
       CQ if "C" in outs else None, csa if "C" in outs else None, G, M, I, ld,
       masked_m=None if masked is None else torch.tensor(masked, dtype=torch.int32, device="cuda"))
    return Y, Q, sa, CQ, csa


def check(GU, got, rows, ue8m0, what):
    Y, Q, sa, CQ, csa = got
    G, M, I2 = GU.shape
    I = I2 // 2
    for z in range(G):
        n = rows[z]
        y, e = R.swiglu(GU[z, :n]), rel(GU)
        R.check_close(Y[z, :n], y, e * y.abs(), f"{what} Y")
        s = (R.unpack_ue8m0(sa[z], n, I // 128) if ue8m0 else R.scales(sa[z], n, I // 128).double())
        R.check_scales(s, y, e, ue8m0, what)
        R.check_codes(Q[z, :n], s, y, 2 * e, what)
        # rows without a token keep what they held
        assert (Y[z, n:] == -3.0).all() and (Q[z, n:] == 0x7F).all() and (CQ[z, n:] == 0x7F).all(), what
        assert (sa[z, :, n:] == (0x55555555 if ue8m0 else -7.25)).all(), what
        assert (csa[z, :, n:] == -7.25).all(), what
    # the checkpoint is the quantiser's output, bit for bit
    wantq, wants = torch.full_like(CQ, 0x7F), torch.full_like(csa, -7.25)
    dg.quantize_fp8_1x128(GU, wantq, wants, G, M, I2, csa.shape[-1])
    for z in range(G):
        n = rows[z]
        assert torch.equal(CQ[z, :n], wantq[z, :n]) and torch.equal(csa[z, :, :n], wants[z, :, :n]), what


@pytest.mark.parametrize("shape", [(1, 1, 128, 4), (1, 37, 256, 40), (1, 200, 2048, 200),
                                   (1, 33, 1536, 36), (1, 1000, 640, 1000)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ue8m0", [False, True])
def test_swiglu(shape, ue8m0):
    G, M, I, ld = shape
    GU = normal(G, M, 2 * I, seed=M + I, scale=2.0)
    check(GU, forward(GU, ld, ue8m0=ue8m0), [M] * G, ue8m0, f"{shape}")
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("masked", [[0, 0, 0], [64, 0, 1], [33, 64, 31], [32, 63, 2]])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_masked_rows(masked, ue8m0):
    GU = normal(3, 64, 512, seed=sum(masked), scale=1.5)
    for z, n in enumerate(masked):
        GU[z, n:] = float("nan")         # what lies there is not read into any output
    check(GU, forward(GU, 68, masked, ue8m0), masked, ue8m0, f"{masked}")
    assert dg.get_device_status() == 0


def test_masked_count_out_of_range_is_clamped_and_reported():
    GU = normal(2, 40, 256, seed=3)
    check(GU, forward(GU, 40, [-3, 41]), [0, 40], False, "clamped")
    assert dg.get_device_status() == 8 and dg.get_device_status() == 0


def test_extreme_values():
    """Large gates of either sign, zeros, groups below the scale's floor."""
    GU = normal(1, 8, 512, seed=5, scale=30.0)
    GU[0, 0] = 0
    GU[0, 1] *= 1e-12
    GU[0, 2, :256] = -120.0              # silu underflows to zero
    GU[0, 3, :256] = 120.0
    GU[0, 4, 256:] = -0.0
    Y, Q, sa, CQ, csa = forward(GU, 8)
    y = R.swiglu(GU)
    # (silu(-87 and below) is lost below the smallest normal fp32 number)
    R.check_close(Y, y, rel(GU) * y.abs() + 2.0 ** -120, "extreme Y")
    R.check_codes(Q, R.scales(sa, 8, 2).double(), y, 2 * rel(GU), "extreme Q")
    assert (Q[0, 0] & 0x7F == 0).all()


@pytest.mark.parametrize("outs", ["Y", "Q", "C", "YC", "QC"])
def test_optional_outputs(outs):
    GU = normal(1, 21, 512, seed=6)
    all_, some = forward(GU, 24), forward(GU, 24, outs=outs)
    Y, Q, sa, CQ, csa = some
    for name, i in (("Y", 0), ("Q", 1), ("Q", 2), ("C", 3), ("C", 4)):
        if name in outs:
            assert torch.equal(some[i], all_[i])
        else:
            assert (some[i] == some[i].view(-1)[0]).all()


def backward(CQ, csa, dY, masked=None, y=True):
    G, M, I2 = CQ.shape
    dGU = torch.full((G, M, I2), -3.0, dtype=torch.bfloat16, device="cuda")
    Y = torch.full((G, M, I2 // 2), -3.0, dtype=torch.bfloat16, device="cuda")
    dg.swiglu_backward_fp8_1x128(
        CQ, csa, dY, dGU, Y if y else None, G, M, I2 // 2, csa.shape[-1],
        masked_m=None if masked is None else torch.tensor(masked, dtype=torch.int32, device="cuda"))
    return dGU, Y


@pytest.mark.parametrize("shape,masked", [((1, 1, 128), None), ((1, 45, 256), None),
                                          ((1, 300, 1536), None), ((3, 64, 384), [64, 0, 33]),
                                          ((2, 31, 2048), [1, 30])])
def test_swiglu_gradient(shape, masked):
    G, M, I = shape
    ld = (M + 3) // 4 * 4 + 4
    GU = normal(G, M, 2 * I, seed=M, scale=2.0)
    dY = normal(G, M, I, seed=M + 1, scale=0.05)
    CQ, csa = torch.zeros(G, M, 2 * I, dtype=torch.uint8, device="cuda"), torch.zeros(
        G, 2 * I // 128, ld, device="cuda")
    dg.quantize_fp8_1x128(GU, CQ, csa, G, M, 2 * I, ld)
    dGU, Y = backward(CQ, csa, dY, masked)
    # the values the checkpoint stands for, in the kernel's fp32 (code * scale)
    gu = (R.groups(CQ.view(torch.float8_e4m3fn).float()) * R.scales(csa, M, 2 * I // 128)[..., None]
          ).flatten(-2)
    y, d = R.swiglu(gu), R.swiglu_backward(gu, dY)
    g, u = gu.double().chunk(2, -1)
    s, dy = torch.sigmoid(g), dY.double()
    e = rel(g)
    mag = torch.cat([(dy * u).abs() * s * (1 + g.abs()), (dy * g * s).abs()], -1)
    for z in range(G):
        n = M if masked is None else masked[z]
        R.check_close(dGU[z, :n], d[z, :n], 2 * e * mag[z, :n], f"{shape} dGU")
        R.check_close(Y[z, :n], y[z, :n], e * y[z, :n].abs(), f"{shape} Y")
        assert (dGU[z, n:] == -3.0).all() and (Y[z, n:] == -3.0).all()
    only, untouched = backward(CQ, csa, dY, masked, y=False)
    assert torch.equal(only, dGU) and (untouched == -3.0).all()
    assert dg.get_device_status() == 0


def test_gradient_from_the_checkpoint_is_near_the_gradient_of_the_input():
    """The checkpoint costs the gradient what 8 bits cost its input: an element
    is off by at most its code's half spacing."""
    GU, dY = normal(1, 128, 1024, seed=9, scale=1.5), normal(1, 128, 512, seed=10)
    _, _, _, CQ, csa = forward(GU, 128)
    dGU, _ = backward(CQ, csa, dY)
    want = R.swiglu_backward(GU, dY)
    # codes are off by 2^-4 of themselves at most, 2^-4 / sqrt(3) or less on
    # average; the gate's gradient multiplies two of them and a smooth factor
    assert (dGU.double() - want).norm() <= 2 * 2.0 ** -4 / 3 ** 0.5 * want.norm()


def test_graph_capture_follows_new_counts():
    GU = normal(2, 32, 512, seed=11)
    mm = torch.tensor([32, 5], dtype=torch.int32, device="cuda")
    Q = torch.full((2, 32, 256), 0x7F, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(2, 2, 32, device="cuda")
    call = lambda: dg.swiglu_quantize_fp8_1x128(GU, None, Q, sa, None, None, 2, 32, 256, 32, masked_m=mm)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    Q.fill_(0x7F)
    mm.copy_(torch.tensor([3, 32], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    assert (Q[0, 3:] == 0x7F).all() and (Q[0, :3] & 0x7F != 0x7F).all() and (Q[1] & 0x7F != 0x7F).all()


def test_rows_past_32_bit_offsets():
    M, I = 600_000, 2048                # GU: 2.4e9 elements
    GU = torch.zeros(1, M, 2 * I, dtype=torch.bfloat16, device="cuda")
    GU[0, -3:] = normal(3, 2 * I, seed=12)
    Q = torch.full((1, M, I), 0x7F, dtype=torch.uint8, device="cuda")
    sa = torch.zeros(1, I // 128, M, device="cuda")
    CQ = torch.full((1, M, 2 * I), 0x7F, dtype=torch.uint8, device="cuda")
    csa = torch.zeros(1, 2 * I // 128, M, device="cuda")
    dg.swiglu_quantize_fp8_1x128(GU, None, Q, sa, CQ, csa, 1, M, I, M)
    y = R.swiglu(GU[0, -3:])
    s = sa[0, :, -3:].t().double()
    R.check_scales(s, y, rel(GU[0, -3:]), False, "tail")
    R.check_codes(Q[0, -3:], s, y, 2 * rel(GU[0, -3:]), "tail")
    assert (Q[0, :-3] == 0).all()
    dY = torch.zeros(1, M, I, dtype=torch.bfloat16, device="cuda")
    dY[0, -3:] = normal(3, I, seed=13)
    del GU, Q
    dGU, _ = backward(CQ, csa, dY, y=False)
    gu = (R.groups(CQ[0, -3:].view(torch.float8_e4m3fn).float()) * csa[0, :, -3:].t()[..., None]).flatten(-2)
    want = R.swiglu_backward(gu, dY[0, -3:])
    assert (dGU[0, -3:].double() - want).norm() <= R.BF16_ROUND * want.norm()
    assert (dGU[0, :-3] == 0).all()
