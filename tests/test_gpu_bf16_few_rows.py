"""The ragged bf16 products of a few rows in all, which have a form of their own,
against their 64-bit definitions."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from tests import operators_ref as R
from tests.test_gpu_bf16_ragged import KEEP, inputs, ints, normal, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from moe_grouped_gemm_bf16_gb300 import _build
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    dg.set_num_sms(0)


def check(form, A, B, sizes, D, what, C=None):
    """fp32 sums in any order: an ulp's half (u) of a partial sum per product and
    joining step (at most 5 shuffles and 16 warps), at most all of the
    magnitudes; one more for the addend."""
    want, mag = R.products(form, A, B, sizes, C)
    length = max(sizes) if form == "tn" else A.shape[1]
    R.check_close(D[:want.shape[0]], want, (length + 22) * R.U32 * mag, what)
    assert (D[want.shape[0]:] == KEEP).all(), f"{what}: rows past the groups were written"
    assert dg.get_device_status() == 0, what


def spread(groups, **rows):
    return [rows.get(f"g{i}", 0) for i in range(groups)]


# one to eight rows in one group (every pass and remainder), alone or behind and
# between groups without any, and more groups than a warp has lanes
SIZES = [[1], [2], [3], [4], [0, 4, 0], [1, 0, 2, 1], spread(33, g0=1, g32=2), spread(100, g40=5, g99=3),
         spread(64, g31=7, g32=1), spread(70, g1=1, g2=1, g35=8, g64=2), [1] * 8 + [0] * 120]
# K below, at and beyond a warp's run of 256 and its splits, N of one vector of 8
# and around the blocks' columns
DIMS = [(8, 8), (16, 264), (72, 248), (136, 2056), (1048, 264), (264, 4104), (2576, 520)]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}g" + "-".join(str(x) for x in s if x))
@pytest.mark.parametrize("dims", DIMS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_few_rows(form, dims, sizes):
    N, K = dims
    if len(sizes) * N * K > 1 << 27:
        sizes = sizes[:1 + max(i for i, s in enumerate(sizes) if s)][-40:]
    A, B = inputs(form, sizes, N, K, seed=N + K)
    check(form, A, B, sizes, run(form, A, B, sizes, N), f"{form} {dims}")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_most_rows_of_one_group(form):
    """As many as the form takes, all in one of many groups."""
    sizes = spread(128, g77=32)
    A, B = inputs(form, sizes, 200, 392, seed=3)
    check(form, A, B, sizes, run(form, A, B, sizes, 200), form)


@pytest.mark.parametrize("sizes", [[0, 3, 1], [0, 0], [8]])
@pytest.mark.parametrize("in_place", [False, True])
def test_addend(sizes, in_place):
    A, B = inputs("tn", sizes, 328, 136, seed=5, rows=max(1, sum(sizes)))
    C = normal(len(sizes), 136, 328, seed=6)
    D = C.clone() if in_place else None
    D = run("tn", A, B, sizes, 328, C=D if in_place else C, D=D)
    check("tn", A, B, sizes, D, "addend", C=C)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_other_values_do_not_leak(form, bad):
    """Rows and weights of other groups, and rows past all groups."""
    sizes = [1, 2, 0, 1]
    A, B = inputs(form, sizes, 136, 520, seed=7, rows=6)
    clean = run(form, A, B, sizes, 136)
    A[1:3] = bad
    A[4:] = bad
    if form == "tn":
        B[4:] = bad
        keep = [0, 2, 3]
    else:
        B[2] = bad
        keep = [0, 3]
    D = run(form, A, B, sizes, 136)
    assert torch.equal(D[keep], clean[keep])
    touched = D[1] if form == "tn" else D[1:3]
    assert not torch.isfinite(touched.float()).all()
    if form != "tn":
        assert (D[4:] == KEEP).all()


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("given,taken", [([1, -4, 2, 0], [1, 0, 2, 0]), ([1, 9, 2, 5], [1, 3, 0, 0]),
                                         ([2 ** 31 - 1, 2 ** 31 - 1, 5, -1], [4, 0, 0, 0]),
                                         ([0] * 40 + [2, 3] + [0] * 30, [0] * 40 + [2, 2] + [0] * 30)])
def test_bad_sizes_are_clamped_and_reported(form, given, taken):
    A, B = inputs(form, taken, 136, 72, seed=29, rows=4)
    D = run(form, A, B, given, 136)
    assert dg.get_device_status() == 10 and dg.get_device_status() == 0
    check(form, A, B, taken, D, f"{form} {given}")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_graph_capture_follows_new_sizes(form):
    sizes, later = [2, 0, 1], [0, 3, 0]
    A, B = inputs(form, sizes, 264, 520, seed=37)
    n = ints(sizes)
    D = run(form, A, B, sizes, 264, dev_sizes=n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(form, A, B, sizes, 264, D=D, dev_sizes=n)
    n.copy_(ints(later))
    D.fill_(KEEP)
    graph.replay()
    torch.cuda.synchronize()
    check(form, A, B, later, D, f"{form} graph")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_same_bits_and_near_the_tiled_form(form):
    """The same inputs give the same bits; a limit on the SMs takes the tiled form."""
    sizes = [1, 3]
    A, B = inputs(form, sizes, 1160, 1032, seed=41)
    first = run(form, A, B, sizes, 1160)
    for _ in range(3):
        assert torch.equal(run(form, A, B, sizes, 1160), first)
    dg.set_num_sms(20)
    try:
        tiled = run(form, A, B, sizes, 1160)
    finally:
        dg.set_num_sms(0)
    check(form, A, B, sizes, first, form)
    check(form, A, B, sizes, tiled, f"{form} tiled")


def test_another_stream():
    """Work queued on a stream before the call is seen by it."""
    s = torch.cuda.Stream()
    A, B = inputs("nt", [1, 1], 512, 1024, seed=43)
    late = torch.empty_like(A)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        late.copy_(A)
        D = run("nt", late, B, [1, 1], 512)
    s.synchronize()
    check("nt", A, B, [1, 1], D, "stream")
