"""The ragged bf16 products on the GPU against their 64-bit definitions."""
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import operators_ref as R

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
    dg.debug_force_ragged_plan()


def normal(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def inputs(form, sizes, N, K, seed=0, rows=None):
    """A, B of the form; for tn, K is the M of D [G, M, N]."""
    T, G = rows or sum(sizes), len(sizes)
    A = normal(T, K, seed=seed + 1)
    if form == "nt":
        return A, normal(G, N, K, seed=seed + 2)
    if form == "nn":
        return A, normal(G, K, N, seed=seed + 2)
    return A, normal(T, N, seed=seed + 2)


def run(form, A, B, sizes, N, C=None, D=None, dev_sizes=None):
    """`sizes` on the device; D starts full of KEEP."""
    T, G = A.shape[0], len(sizes)
    n = ints(sizes) if dev_sizes is None else dev_sizes
    if form == "tn":
        D = torch.full((G, A.shape[1], N), KEEP, dtype=torch.bfloat16, device="cuda") if D is None else D
        dg.k_grouped_gemm_bf16_tn_ragged(A, B, D, n, G, A.shape[1], N, T, C=C)
    else:
        D = torch.full((T, N), KEEP, dtype=torch.bfloat16, device="cuda") if D is None else D
        fn = dg.m_grouped_gemm_bf16_nt_ragged if form == "nt" else dg.m_grouped_gemm_bf16_nn_ragged
        fn(A, B, D, n, T, N, A.shape[1], G)
    return D


def check(form, A, B, sizes, D, what, C=None):
    """fp32 sums: each of the (length / 16) steps of the tensor cores loses at
    most an ulp (two u) of a partial sum, doubled for what a step itself loses."""
    want, mag = R.products(form, A, B, sizes, C)
    length = max(sizes) if form == "tn" else A.shape[1]
    slack = (length / 16 + 4) * 4 * R.U32 * mag
    R.check_close(D[:want.shape[0]], want, slack, what)
    assert (D[want.shape[0]:] == KEEP).all(), f"{what}: rows past the groups were written"
    assert dg.get_device_status() == 0, what


SIZES = [[1], [16], [5, 0, 3], [0, 0, 70], [64, 64], [129, 1, 0, 255], [300, 17, 256], [31] * 40,
         [0, 513, 2, 0]]
DIMS = [(128, 64), (8, 8), (136, 72), (200, 328), (256, 128), (392, 520)]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s[:5])))
@pytest.mark.parametrize("dims", DIMS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_product(form, dims, sizes):
    N, K = dims
    A, B = inputs(form, sizes, N, K, seed=sum(sizes) + N)
    check(form, A, B, sizes, run(form, A, B, sizes, N), f"{form} {dims} {sizes}")


@pytest.mark.parametrize("form,sizes,N,K", [
    ("nt", [700, 1, 1300, 0, 520], 1024, 1536), ("nn", [700, 1, 1300, 0, 520], 1032, 1544),
    ("tn", [700, 1, 1300, 0, 520], 1024, 1536), ("tn", [900, 0, 77], 776, 1032),
    ("nt", [6] * 8, 4096, 2048), ("nt", [61], 2112, 7168), ("nn", [3, 0, 1, 9], 2048, 1024),
    ("nt", [1], 7168, 2048), ("nn", [1, 0], 7168, 2048), ("tn", [4097], 264, 520),
    ("tn", [20000], 128, 256),
    # few tiles: the reduction split over a cluster, with uneven and empty shares
    ("nt", [1], 64, 8192), ("nt", [5, 0], 72, 4168), ("nn", [33], 128, 6000), ("nn", [2], 64, 1160),
    ("nt", [300], 256, 8192), ("nn", [170, 180], 264, 5000), ("tn", [3000, 0, 20], 64, 128),
    ("tn", [5001, 7], 256, 264), ("tn", [8000], 520, 40), ("nt", [100], 200, 7176)])
def test_larger_products(form, sizes, N, K):
    A, B = inputs(form, sizes, N, K, seed=7)
    check(form, A, B, sizes, run(form, A, B, sizes, N), f"{form} {sizes}")


PLANS = [(True, 256, 256, s) for s in (1, 2, 4)] + [
    (False, l, r, s) for l, r, s in ((64, 16, 1), (64, 64, 8), (112, 48, 1), (128, 64, 3), (128, 128, 1),
                                     (192, 16, 5), (192, 128, 1), (256, 64, 2), (256, 128, 8))]


@pytest.mark.parametrize("plan", PLANS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_every_tiling(form, plan):
    """Every kernel form on the same ragged shapes: edges of lanes, rows and
    reduction, shares of the reduction without a slot, groups without rows."""
    dg.debug_force_ragged_plan(*plan)
    try:
        for sizes, N, K in (([5, 0, 300, 33], 264, 392), ([130, 257, 0], 520, 1032), ([70], 200, 64),
                            ([17, 16, 1], 328, 2056)):
            A, B = inputs(form, sizes, N, K, seed=sum(sizes))
            check(form, A, B, sizes, run(form, A, B, sizes, N), f"{form} {plan} {sizes}")
        if form == "tn":
            C = normal(4, 392, 264, seed=51)
            A, B = inputs(form, [5, 0, 300, 33], 264, 392, seed=52)
            check(form, A, B, [5, 0, 300, 33], run(form, A, B, [5, 0, 300, 33], 264, C=C),
                  f"addend {plan}", C=C)
    except dg.DGError as e:
        # (a 64-wide box where the forced tile is narrower: refused, not wrong)
        assert e.status == 2 and not plan[0] and (plan[1] % 64 or (form == "tn" and plan[2] % 64))
    finally:
        dg.debug_force_ragged_plan()


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_many_groups(form):
    g = torch.Generator().manual_seed(3)
    sizes = torch.randint(0, 4, (1024,), generator=g).tolist()
    A, B = inputs(form, sizes, 64, 72, seed=11)
    check(form, A, B, sizes, run(form, A, B, sizes, 64), f"{form} 1024 groups")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("sms", [1, 3])
def test_few_sms(form, sms):
    """Every CTA takes many tiles (both accumulators, every ring phase)."""
    sizes = [300, 0, 41, 513]
    A, B = inputs(form, sizes, 520, 456, seed=13)
    dg.set_num_sms(sms)
    try:
        D = run(form, A, B, sizes, 520)
    finally:
        dg.set_num_sms(0)
    check(form, A, B, sizes, D, f"{form} on {sms} SMs")


@pytest.mark.parametrize("form", ["nt", "nn"])
def test_rows_past_the_groups_are_not_written(form):
    sizes = [20, 0, 37]
    A, B = inputs(form, sizes, 136, 200, seed=17, rows=100)
    check(form, A, B, sizes, run(form, A, B, sizes, 136), f"{form} partly filled")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_other_groups_values_do_not_leak(form, bad):
    """What one group's rows (or the rows past all groups) hold, NaN and
    infinities among it, reaches no other group's result."""
    sizes = [21, 50, 33]
    A, B = inputs(form, sizes, 264, 136, seed=19, rows=120)
    clean = [A[:21].clone(), A[71:104].clone()]
    A[21:71] = bad
    A[104:] = bad
    if form == "tn":
        B[21:71] = bad
        B[104:] = bad
    D = run(form, A, B, sizes, 264)
    want, mag = R.products(form, A, B, sizes)
    pick = [0, 2] if form == "tn" else list(range(21)) + list(range(71, 104))
    assert torch.isfinite(want[pick]).all()
    R.check_close(D[pick], want[pick], 16 * 4 * R.U32 * mag[pick], f"{form} leak")
    assert not torch.isfinite(D[[1] if form == "tn" else [30]]).any()
    assert dg.get_device_status() == 0


def test_values_that_overflow_bf16_become_infinite():
    A, B = torch.full((3, 64), 1e30, device="cuda").bfloat16(), torch.full(
        (1, 128, 64), 1e9, device="cuda").bfloat16()
    D = run("nt", A, B, [3], 128)
    assert torch.isinf(D).all() and (D > 0).all()


@pytest.mark.parametrize("sizes", [[70, 0, 9], [0, 0, 0], [16, 32, 48]])
@pytest.mark.parametrize("in_place", [False, True])
def test_addend(sizes, in_place):
    M, N = 200, 136
    A, B = inputs("tn", sizes, N, M, seed=23, rows=sum(sizes) + 1)
    C = normal(len(sizes), M, N, seed=24, scale=5.0)
    keep = C.clone()
    D = run("tn", A, B, sizes, N, C=C, D=C if in_place else None)
    check("tn", A, B, sizes, D, f"addend {sizes}", C=keep)
    for g, n in enumerate(sizes):
        if n == 0:
            assert torch.equal(D[g], keep[g])


def test_gradient_without_any_rows():
    for C in (None, normal(2, 64, 72, seed=25)):
        D = torch.full((2, 64, 72), KEEP, dtype=torch.bfloat16, device="cuda")
        dg.k_grouped_gemm_bf16_tn_ragged(None, None, D, ints([0, 0]), 2, 64, 72, 0, C=C)
        assert torch.equal(D, torch.zeros_like(D) if C is None else C)
    assert dg.get_device_status() == 0


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
@pytest.mark.parametrize("given,taken", [([30, -4, 20], [30, 0, 20]), ([30, 90, 20], [30, 50, 0]),
                                         ([2 ** 31 - 1, 2 ** 31 - 1, 5], [80, 0, 0])])
def test_bad_sizes_are_clamped_and_reported(form, given, taken):
    A, B = inputs(form, taken, 136, 72, seed=29, rows=80)
    if form != "tn":
        B = B[:3]
    D = run(form, A, B, given, 136)
    assert dg.get_device_status() == 10 and dg.get_device_status() == 0
    check(form, A, B, taken, D, f"{form} {given}")


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_same_inputs_same_bits(form):
    sizes = [333, 5, 0, 90]
    A, B = inputs(form, sizes, 776, 904, seed=31)
    first = run(form, A, B, sizes, 776)
    for _ in range(3):
        assert torch.equal(run(form, A, B, sizes, 776), first)


@pytest.mark.parametrize("form", ["nt", "nn", "tn"])
def test_graph_capture_follows_new_sizes(form):
    sizes, later = [40, 0, 24], [0, 60, 4]
    A, B = inputs(form, sizes, 264, 200, seed=37)
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


def test_two_streams_at_once():
    sizes = [200, 30]
    A, B = inputs("nt", sizes, 512, 1024, seed=41)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    torch.cuda.synchronize()
    for s in streams:
        with torch.cuda.stream(s):
            outs += [run("nt", A, B, sizes, 512) for _ in range(4)]
    torch.cuda.synchronize()
    for D in outs:
        check("nt", A, B, sizes, D, "two streams")


@pytest.mark.parametrize("plan", [(False, 0, 0, 1), (True, 256, 256, 1), (True, 256, 256, 4),
                                  (False, 128, 64, 4)], ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("form", ["nt", "tn"])
def test_waits_that_run_out_are_reported(form, plan):
    """With the TMA producer switched off and a short limit every wait gives up,
    the call reports it, and the next call is right again."""
    sizes = [40, 24]
    A, B = inputs(form, sizes, 256, 128, seed=43)
    dg.debug_force_ragged_plan(*plan)
    dg.set_wait_timeout_ns(20_000_000)
    dg.debug_set_skip_producer(True)
    try:
        run(form, A, B, sizes, 256)
        assert dg.get_device_status() == 7
    finally:
        dg.debug_set_skip_producer(False)
        dg.set_wait_timeout_ns(0)
    try:
        check(form, A, B, sizes, run(form, A, B, sizes, 256), f"{form} after a timeout")
    finally:
        dg.debug_force_ragged_plan()


def test_offsets_past_32_bits():
    """D and a weight tensor of more than 2^31 elements."""
    N, T = 32768, 70_000
    A = torch.zeros(T, 64, dtype=torch.bfloat16, device="cuda")
    A[-40:] = normal(40, 64, seed=47)
    B = normal(2, N, 64, seed=48)
    sizes = [T - 20, 20]
    D = run("nt", A, B, sizes, N)
    x = A[-40:].double()
    want = torch.cat([x[:20] @ B[0].double().t(), x[20:] @ B[1].double().t()])
    mag = torch.cat([x[:20].abs() @ B[0].double().abs().t(), x[20:].abs() @ B[1].double().abs().t()])
    R.check_close(D[-40:], want, 8 * 4 * R.U32 * mag, "large D")
    assert (D[:T - 40] == 0).all()
    del D
    W = torch.zeros(9, 16384, 16384, dtype=torch.bfloat16, device="cuda")
    W[-1] = normal(16384, 16384, seed=49)
    x = normal(3, 16384, seed=50)
    sizes = [0] * 8 + [3]
    for form in ("nt", "nn"):
        D = run(form, x, W, sizes, 16384)
        w = W[-1].double().t() if form == "nt" else W[-1].double()
        mag = x.double().abs() @ w.abs()
        R.check_close(D, x.double() @ w, (1024 + 4) * 4 * R.U32 * mag, "large weights")


def test_matches_the_checked_build(tmp_path):
    """The checked library (bounds checks before loads and stores) runs the same
    cases clean."""
    import os
    import subprocess
    import sys
    _build.build(debug=True)
    code = (
        "import torch, moe_grouped_gemm_bf16_gb300 as dg\n"
        "from tests import test_gpu_bf16_ragged as T\n"
        "for form in ('nt', 'nn', 'tn'):\n"
        "    for sizes, N, K in (([5, 0, 3], 136, 72), ([300, 17, 256], 392, 520), ([31] * 40, 128, 64)):\n"
        "        A, B = T.inputs(form, sizes, N, K)\n"
        "        for plan in [()] + T.PLANS:\n"
        "            dg.debug_force_ragged_plan(*plan)\n"
        "            try: D = T.run(form, A, B, sizes, N)\n"
        "            except dg.DGError as e: assert e.status == 2, e; continue\n"
        "            T.check(form, A, B, sizes, D, form)\n"
        "assert dg.lib()._name.endswith('libdg_debug.so')\nprint('checked ok')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, DG_DEBUG="1"),
                         capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and "checked ok" in out.stdout, out.stdout[-2000:] + out.stderr[-3000:]
