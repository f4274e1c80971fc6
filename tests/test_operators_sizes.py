"""Sizes near 2^31 of the ragged bf16 products: the kernels' 32-bit counters step
past an extent before they stop, so an extent within a step of 2^31 would wrap
around and be read or written out of range.  Such calls are refused on the host
(no GPU needed, and none is used: the addresses are made up)."""
import pytest

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests.test_operators_abi import GRAD, ROWS, SHAPE, status

TOP = 2 ** 31 - 8192   # the first multiple of 8 that is refused


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()


@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("kw", [dict(M_total=2 ** 31 - 1, N=8, K=8), dict(M_total=TOP, N=8, K=8),
                                dict(M_total=1, N=8, K=2 ** 31 - 8), dict(M_total=64, N=8, K=2 ** 31 - 8),
                                dict(M_total=1, N=8, K=TOP)])
def test_rows_and_depth(form, kw):
    call = getattr(dg, f"m_grouped_gemm_bf16_{form}_ragged")
    assert status(call, {**ROWS, "num_groups": 1, **kw}) == SHAPE
    # (sizes a step below pass the host's checks: see the next test)


@pytest.mark.parametrize("kw", [dict(K_total=2 ** 31 - 1, M=8, N=8), dict(K_total=TOP, M=8, N=8),
                                dict(K_total=8, M=2 ** 31 - 8, N=8), dict(K_total=8, M=TOP, N=8)])
def test_gradient(kw):
    assert status(dg.k_grouped_gemm_bf16_tn_ragged, {**GRAD, "num_groups": 1, **kw}) == SHAPE


def furthest(extent, step):
    """The largest value that `for (x = x0; x < extent; x += step)` reaches."""
    return extent - 1 + step


@pytest.mark.parametrize("step", [
    2 * 8 * 256,        # few rows, nt: two runs of 256 for each of 8 shares of K
    8 * 512 // 2,       # few rows, nn: 8 rows of B for each of 256 chains
    128 + 128,          # tiles: a slot's depth and both of its pieces
    256 + 128,          # rows of a tile and the second CTA's half
])
def test_counters_of_sizes_that_pass_stay_in_32_bits(step):
    assert furthest(TOP - 8, step) < 2 ** 31
