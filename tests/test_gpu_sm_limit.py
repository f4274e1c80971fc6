"""A limit on the SMs bounds what the operators around the GEMMs launch: every
grid of at most as many blocks as SMs, results as without it."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import test_gpu_bf16_ragged as P
from tests.launches import launched
from tests.test_gpu_bf16_ragged import ints

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
