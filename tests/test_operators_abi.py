"""Refusals of the operators around the FP8 GEMMs: arguments are checked on the
host before a device is touched (no GPU needed)."""
import pytest

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build

P = 0x10000   # a fake, aligned "device" address; never dereferenced
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


def status(fn, kw):
    try:
        fn(**kw)
    except dg.DGError as e:
        assert dg.lib().dg_last_error_string().decode() != ""
        return e.status
    return OK


NORM = dict(X=P, R=P, W=P, H=P, Y=P, Q=P, rstd=P, M=8, K=512, eps=1e-6)
NORM_CASES = [
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(Y=None, Q=None), INVALID),
    (dict(R=None), INVALID), (dict(M=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(K=0), SHAPE), (dict(K=500), SHAPE),
    (dict(K=16384 + 128), SHAPE), (dict(X=P + 8), MISALIGNED), (dict(R=P + 2), MISALIGNED),
    (dict(H=P + 4), MISALIGNED), (dict(Y=P + 8), MISALIGNED), (dict(Q=P + 8), MISALIGNED),
    (dict(rstd=P + 2), MISALIGNED), (dict(M=0), OK), (dict(M=0, R=None, H=None), OK),
]


@pytest.mark.parametrize("kw,code", NORM_CASES)
@pytest.mark.parametrize("ue8m0", [False, True])
def test_norm_refusals(kw, code, ue8m0):
    fn = dg.rms_norm_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.rms_norm_quantize_fp8_1x128
    s, ld = ("sfa", "ld_sfa") if ue8m0 else ("sa", "ld_sa")
    assert status(fn, {**NORM, s: P, ld: 8, **kw}) == code


@pytest.mark.parametrize("kw,code", [
    (dict(sa=None), INVALID), (dict(ld_sa=4), INVALID), (dict(ld_sa=10), MISALIGNED),
    (dict(sa=P + 4), MISALIGNED), (dict(Q=None, sa=None, ld_sa=0, M=0), OK)])
def test_norm_scale_refusals(kw, code):
    assert status(dg.rms_norm_quantize_fp8_1x128, {**NORM, "sa": P, "ld_sa": 8, **kw}) == code


def test_norm_gradient_workspace():
    assert dg.rms_norm_backward_workspace_bytes(0, 512) == 0
    assert dg.rms_norm_backward_workspace_bytes(3, 512) == 3 * 512 * 4
    big = dg.rms_norm_backward_workspace_bytes(10 ** 6, 16384)
    assert big == dg.rms_norm_backward_workspace_bytes(10 ** 9, 16384) and big <= 64 << 20
    assert dg.rms_norm_backward_workspace_bytes(-1, 512) == -1


NORM_BWD = dict(dY=P, H=P, rstd=P, W=P, dR=P, dX=P, dW=P, workspace=P, workspace_bytes=1 << 30, M=8,
                K=512)


@pytest.mark.parametrize("kw,code", [
    (dict(dY=None), INVALID), (dict(H=None), INVALID), (dict(rstd=None), INVALID),
    (dict(W=None), INVALID), (dict(dX=None), INVALID), (dict(dW=None), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace_bytes=100), INVALID), (dict(M=-1), INVALID),
    (dict(K=100), SHAPE), (dict(K=32768), SHAPE), (dict(dY=P + 8), MISALIGNED),
    (dict(dR=P + 8), MISALIGNED), (dict(dW=P + 4), MISALIGNED), (dict(workspace=P + 4), MISALIGNED)])
def test_norm_gradient_refusals(kw, code):
    assert status(dg.rms_norm_backward, {**NORM_BWD, **kw}) == code


SWIGLU = dict(GU=P, Y=P, Q=P, CQ=P, csa=P, num_groups=2, M=8, I=256, masked_m=P)


@pytest.mark.parametrize("kw,code", [
    (dict(GU=None), INVALID), (dict(Y=None, Q=None, CQ=None, csa=None), INVALID),
    (dict(csa=None), INVALID), (dict(CQ=None), INVALID), (dict(num_groups=0), INVALID),
    (dict(M=-1), INVALID), (dict(I=0), SHAPE), (dict(I=200), SHAPE), (dict(num_groups=65536), SHAPE),
    (dict(I=128 * 32768), SHAPE), (dict(GU=P + 8), MISALIGNED), (dict(Y=P + 2), MISALIGNED),
    (dict(CQ=P + 8), MISALIGNED), (dict(csa=P + 4), MISALIGNED), (dict(masked_m=P + 2), MISALIGNED),
    (dict(M=0), OK)])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_swiglu_refusals(kw, code, ue8m0):
    fn = dg.swiglu_quantize_fp8_1x128_ue8m0 if ue8m0 else dg.swiglu_quantize_fp8_1x128
    s, ld = ("sfa", "ld_sfa") if ue8m0 else ("sa", "ld_sa")
    assert status(fn, {**SWIGLU, s: P, ld: 8, **kw}) == code


@pytest.mark.parametrize("kw,code", [
    (dict(sa=None), INVALID), (dict(ld_sa=4), INVALID), (dict(ld_sa=9), MISALIGNED)])
def test_swiglu_scale_refusals(kw, code):
    assert status(dg.swiglu_quantize_fp8_1x128, {**SWIGLU, "sa": P, "ld_sa": 8, **kw}) == code


SWIGLU_BWD = dict(CQ=P, csa=P, dY=P, dGU=P, Y=P, num_groups=2, M=8, I=256, ld_csa=8, masked_m=P)


@pytest.mark.parametrize("kw,code", [
    (dict(CQ=None), INVALID), (dict(csa=None), INVALID), (dict(dY=None), INVALID),
    (dict(dGU=None), INVALID), (dict(num_groups=0), INVALID), (dict(M=-1), INVALID),
    (dict(ld_csa=4), INVALID), (dict(I=64), SHAPE), (dict(ld_csa=10), MISALIGNED),
    (dict(dGU=P + 8), MISALIGNED), (dict(Y=P + 8), MISALIGNED), (dict(M=0), OK)])
def test_swiglu_gradient_refusals(kw, code):
    assert status(dg.swiglu_backward_fp8_1x128, {**SWIGLU_BWD, **kw}) == code


ROWS = dict(A=P, B=P, D=P, ms=P, M_total=64, N=128, K=256, num_groups=4)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(D=None), INVALID),
    (dict(ms=None), INVALID), (dict(M_total=-1), INVALID), (dict(num_groups=0), INVALID),
    (dict(num_groups=1025), INVALID), (dict(N=0), SHAPE), (dict(N=100), SHAPE), (dict(K=0), SHAPE),
    (dict(K=12), SHAPE), (dict(A=P + 8), MISALIGNED), (dict(D=P + 2), MISALIGNED),
    (dict(ms=P + 2), MISALIGNED), (dict(M_total=0), OK),
    (dict(M_total=2 ** 31 - 1, N=2 ** 20, K=8), SHAPE)])
@pytest.mark.parametrize("form", ["nt", "nn"])
def test_ragged_product_refusals(form, kw, code):
    assert status(getattr(dg, f"m_grouped_gemm_bf16_{form}_ragged"), {**ROWS, **kw}) == code


GRAD = dict(A=P, B=P, C=P, D=P, ks=P, num_groups=4, M=64, N=128, K_total=256)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(D=None), INVALID),
    (dict(ks=None), INVALID), (dict(K_total=-1), INVALID), (dict(num_groups=1025), INVALID),
    (dict(M=12), SHAPE), (dict(N=12), SHAPE), (dict(C=P + 8), MISALIGNED), (dict(B=P + 4), MISALIGNED),
    (dict(M=0), OK)])
def test_ragged_gradient_refusals(kw, code):
    assert status(dg.k_grouped_gemm_bf16_tn_ragged, {**GRAD, **kw}) == code


@pytest.mark.parametrize("plan,code", [
    ((True, 256, 256, 1), OK), ((True, 128, 256, 1), INVALID), ((True, 256, 256, 8), INVALID),
    ((False, 32, 64, 1), INVALID), ((False, 264, 64, 1), INVALID), ((False, 128, 136, 1), INVALID),
    ((False, 128, 64, 9), INVALID), ((False, 128, 64, 0), INVALID), ((False, 0, 0, 0), OK)])
def test_forced_plan_refusals(plan, code):
    try:
        assert status(lambda: dg.debug_force_ragged_plan(*plan), {}) == code
    finally:
        dg.debug_force_ragged_plan()


class Tensor:
    def __init__(self, address):
        self.address = address

    def data_ptr(self):
        if isinstance(self.address, Exception):
            raise self.address
        return self.address


@pytest.mark.parametrize("kw,error", [
    (dict(X=1.5), AttributeError), (dict(X=Tensor(1.5)), TypeError),
    (dict(X=Tensor(KeyError("x"))), KeyError), (dict(X=1 << 70), OverflowError),
    (dict(M=2.0), TypeError), (dict(M=None), TypeError), (dict(M=1 << 31), OverflowError),
    (dict(M=-(1 << 31) - 1), OverflowError), (dict(K=1 << 70), OverflowError),
    (dict(eps="small"), TypeError), (dict(rstd="x"), AttributeError)])
def test_arguments_of_other_types(kw, error):
    with pytest.raises(error):
        dg.rms_norm_quantize_fp8_1x128(**{**NORM, "sa": P, "ld_sa": 8, **kw})


def test_arguments_reach_the_entry_points():
    # tensors, addresses, None; whole numbers of other types; a stream's address
    class Eight:
        def __index__(self):
            return 8
    kw = {**NORM, "sa": Tensor(P), "ld_sa": Eight(), "X": Tensor(P), "M": Eight(), "eps": 1}
    assert status(dg.rms_norm_quantize_fp8_1x128, {**kw, "W": Tensor(0)}) == INVALID
    assert status(dg.rms_norm_quantize_fp8_1x128, {**kw, "W": Tensor(P + 8)}) == MISALIGNED
    assert status(dg.rms_norm_quantize_fp8_1x128, {**kw, "M": 0, "stream": P}) == OK


@pytest.mark.parametrize("given", [0, 12, 14])
def test_number_of_arguments(given):
    from moe_grouped_gemm_bf16_gb300 import _binding
    dg.lib()
    with pytest.raises(TypeError, match="takes 13 arguments"):
        _binding.rms_norm_quantize_fp8_1x128(*[0] * given)
