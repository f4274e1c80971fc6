"""The ragged bf16 products of as many groups as the tables in shared memory leave room
for beside the slots of a CTA pair: seven of 32 KB up to 219 groups."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests.launches import launched
from tests.test_gpu_bf16_ragged import check, inputs, ints, run

pytestmark = pytest.mark.gpu

SLOT = 32768        # 128 lanes and 128 rows, 64 deep, in bf16
LAUNCH = 232448     # the most shared memory of a block


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    dg.debug_force_ragged_plan()
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("groups", [1, 215, 216, 219, 220])
def test_slots_of_a_pair(form, groups):
    sizes = [3 + (g % 5) for g in range(groups)]
    A, B = inputs(form, sizes, 256, 192)
    dg.debug_force_ragged_plan(True, 256, 256, 1)
    try:
        D = run(form, A, B, sizes, 256)
        check(form, A, B, sizes, D, f"{form} of {groups} groups")
        n = ints(sizes)
        if form == "tn":
            call = lambda s: dg.k_grouped_gemm_bf16_tn_ragged(A, B, D, n, groups, 192, 256, A.shape[0], stream=s)
        else:
            fn = dg.m_grouped_gemm_bf16_nt_ragged if form == "nt" else dg.m_grouped_gemm_bf16_nn_ragged
            call = lambda s: fn(A, B, D, n, A.shape[0], 256, 192, groups, stream=s)
        (_, _, smem), = launched(call)
    finally:
        dg.debug_force_ragged_plan()
    assert smem <= LAUNCH
    assert smem // SLOT == (7 if groups <= 219 else 6)
