"""The forms of the gated activation and of the norm that keep a ring of
bulk-copied rows in shared memory: their results over the shapes that reach
them, and what they do when a wait gives up."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import operators_ref as R
from tests.launches import launched
from tests.test_gpu_swiglu import normal, rel

pytestmark = pytest.mark.gpu

KEEP = -3.0


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    dg.debug_set_skip_producer(False)
    dg.set_wait_timeout_ns(0)
    dg.set_num_sms(0)


class Activation:
    """Inputs and outputs of one call (outputs full of what must not stay)."""

    def __init__(self, G, M, I, ue8m0, outs, seed):
        self.G, self.M, self.I, self.ue8m0, self.outs = G, M, I, ue8m0, outs
        self.ld = (M + 3) // 4 * 4
        self.GU = normal(G, M, 2 * I, seed=seed, scale=1.5)
        self.Y = torch.full((G, M, I), KEEP, dtype=torch.bfloat16, device="cuda")
        self.Q = torch.full((G, M, I), 0x7F, dtype=torch.uint8, device="cuda")
        self.sa = (torch.full((G, (I + 511) // 512, self.ld), 0x55555555, dtype=torch.int32, device="cuda")
                   if ue8m0 else torch.full((G, I // 128, self.ld), -7.25, device="cuda"))
        self.CQ = torch.full((G, M, 2 * I), 0x7F, dtype=torch.uint8, device="cuda")
        self.csa = torch.full((G, 2 * I // 128, self.ld), -7.25, device="cuda")

    def __call__(self, stream=None):
        on = lambda x, o: x if o in self.outs else None
        fn = dg.swiglu_quantize_fp8_1x128_ue8m0 if self.ue8m0 else dg.swiglu_quantize_fp8_1x128
        fn(self.GU, on(self.Y, "Y"), on(self.Q, "Q"), on(self.sa, "Q"), on(self.CQ, "C"),
           on(self.csa, "C"), self.G, self.M, self.I, self.ld, stream=stream)

    def check(self):
        M, I, e = self.M, self.I, rel(self.GU)
        for z in range(self.G):
            y = R.swiglu(self.GU[z])
            if "Y" in self.outs:
                R.check_close(self.Y[z], y, e * y.abs(), "Y")
            if "Q" in self.outs:
                s = (R.unpack_ue8m0(self.sa[z], M, I // 128) if self.ue8m0
                     else R.scales(self.sa[z], M, I // 128).double())
                R.check_scales(s, y, e, self.ue8m0, "sa")
                R.check_codes(self.Q[z], s, y, 2 * e, "Q")
                assert (self.sa[z, :, M:] == (0x55555555 if self.ue8m0 else -7.25)).all()
        assert "Y" in self.outs or (self.Y == KEEP).all()
        assert "Q" in self.outs or (self.Q == 0x7F).all()
        if "C" in self.outs:
            # the checkpoint is the quantiser's output, bit for bit
            q, s = torch.empty_like(self.CQ), torch.full_like(self.csa, -7.25)
            dg.quantize_fp8_1x128(self.GU, q, s, self.G, M, 2 * I, self.ld)
            assert torch.equal(self.CQ, q) and torch.equal(self.csa, s)
        else:
            assert (self.CQ == 0x7F).all()
        assert dg.get_device_status() == 0


# groups, rows, width, SMs (0: all).  On all SMs a block's chunk is 48 KB; rows
# that are no multiple of a chunk's, groups that end inside one, rows of more
# lanes than a block has threads, every slot filled several times.
SHAPES = [(1, 11003, 2048, 0), (1, 34700, 640, 0), (3, 3651, 2048, 0), (1, 1833, 8192, 0),
          (1, 175200, 128, 0), (2, 1831, 6144, 0),
          (1, 2701, 128, 1), (1, 601, 640, 1), (1, 401, 2048, 2), (5, 83, 2048, 2), (3, 47, 4224, 3),
          (1, 151, 8192, 2), (1, 60, 16384, 2)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ue8m0,outs", [(False, "QC"), (True, "YQC"), (False, "YC"), (True, "QC")])
def test_ring_with_checkpoint(shape, ue8m0, outs):
    G, M, I, sms = shape
    a = Activation(G, M, I, ue8m0, outs, seed=M + I)
    dg.set_num_sms(sms)
    try:
        a()
        grids = launched(a)
    finally:
        dg.set_num_sms(0)
    assert len(grids) == 1 and grids[0][2] > 0, "not the ring form"
    a.check()


@pytest.mark.parametrize("shape", [(1, 25603, 2048, 0), (2, 2201, 8192, 0), (1, 2701, 128, 1),
                                   (3, 199, 2048, 2)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("ue8m0,outs", [(False, "Q"), (True, "YQ"), (False, "Y")])
def test_ring_without_checkpoint(shape, ue8m0, outs):
    G, M, I, sms = shape
    a = Activation(G, M, I, ue8m0, outs, seed=M + I)
    dg.set_num_sms(sms)
    try:
        a()
        grids = launched(a)
    finally:
        dg.set_num_sms(0)
    assert len(grids) == 1 and grids[0][2] > 0, "not the ring form"
    a.check()


def test_ring_repeats_itself():
    a = Activation(1, 11003, 2048, False, "YQC", seed=3)
    a()
    first = [t.clone() for t in (a.Y, a.Q, a.sa, a.CQ, a.csa)]
    for _ in range(3):
        a()
        assert all(torch.equal(x, y) for x, y in zip(first, (a.Y, a.Q, a.sa, a.CQ, a.csa)))


class no_loads:
    """Inside, the rings' loads are switched off and waits give up after 20 ms."""

    def __enter__(self):
        torch.cuda.synchronize()
        dg.set_wait_timeout_ns(20_000_000)
        dg.debug_set_skip_producer(True)

    def __exit__(self, *unused):
        torch.cuda.synchronize()
        dg.debug_set_skip_producer(False)
        dg.set_wait_timeout_ns(0)


@pytest.mark.parametrize("ue8m0", [False, True])
@pytest.mark.parametrize("sms", [0, 2])
def test_activation_whose_waits_run_out(ue8m0, sms):
    """Every block gives up and ends, nothing is written, the call is reported,
    and the next one is right."""
    a = Activation(1, 11003, 2048, ue8m0, "YQC", seed=5)
    outs = [a.Y, a.Q, a.sa, a.CQ, a.csa]
    before = [t.clone() for t in outs]
    dg.set_num_sms(sms)
    try:
        with no_loads():
            a()
            assert dg.get_device_status() == 7
        assert all(torch.equal(x, y) for x, y in zip(outs, before))
        a()
    finally:
        dg.set_num_sms(0)
    a.check()


@pytest.mark.parametrize("K,M", [(7168, 40), (16384, 30)])
def test_norm_whose_waits_run_out(K, M):
    """The same of the norm's ring, more rows than its slots, H in place of R."""
    X, Rs, W = normal(M, K, seed=1), normal(M, K, seed=2, scale=3.0), normal(K, seed=3)
    keep = Rs.clone()
    Y = torch.full((M, K), KEEP, dtype=torch.bfloat16, device="cuda")
    call = lambda: dg.rms_norm_quantize_fp8_1x128(X, Rs, W, Rs, Y, None, None, None, M, K, 0, 1e-6)
    dg.set_num_sms(1)
    try:
        with no_loads():
            call()
            assert dg.get_device_status() == 7
        assert torch.equal(Rs, keep) and (Y == KEEP).all()
        call()
    finally:
        dg.set_num_sms(0)
    h, _, y = R.norm(X, keep, W, 1e-6)
    R.check_close(Rs, h, R.U32 * h.abs(), "H")
    R.check_close(Y, y, 2.0 ** -18 * y.abs(), "Y")
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("K,M", [(7168, 2000), (1024, 2000), (16384, 470)])
def test_norm_gradient_whose_waits_run_out(K, M):
    dY, H, W = normal(M, K, seed=4, scale=0.03), normal(M, K, seed=5), normal(K, seed=6)
    rstd = torch.rsqrt(H.float().square().mean(-1) + 1e-6)
    n = dg.rms_norm_backward_workspace_bytes(M, K)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    dX = torch.full((M, K), KEEP, dtype=torch.bfloat16, device="cuda")
    dW = torch.empty(K, device="cuda")
    call = lambda: dg.rms_norm_backward(dY, H, rstd, W, None, dX, dW, work, n, M, K)
    with no_loads():
        call()
        assert dg.get_device_status() == 7
    assert (dX == KEEP).all()
    call()
    dx, _ = R.norm_backward(dY, H, rstd, W, None)
    xh, g = H.double() * rstd.double()[:, None], dY.double() * W.double()
    mag = rstd.double()[:, None] * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    R.check_close(dX, dx, 2.0 ** -18 * mag, "dX")
    assert dg.get_device_status() == 0
