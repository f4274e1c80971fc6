"""The experts' rows, dispatch and combine against their definitions in 64 bits.

Bounds.  Rows, sizes and what is copied are exact.  A sum of n products in fp32:
(n + 1) 2^-24 of the sum over magnitudes, and one rounding to bf16 (2^-8 of the
value).  A dot product of K terms over a block: each thread adds K / 32 / 8 terms
at least, (K / 8 + 16) 2^-24 of the sum over magnitudes covers any order of them."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_bf16_gb300 as dg
from moe_grouped_gemm_bf16_gb300 import _build
from tests import moe_ref as M
from tests import operators_ref as R
from tests.launches import launched

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF16 = torch.bfloat16
KEEP = -7.0   # what no call may write


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    torch.cuda.init()
    dg.get_device_status()
    yield
    assert dg.get_device_status() == 0


def choices(T, G, k, seed, empty=0.1, skew=False):
    rng = np.random.default_rng(seed)
    p = (1.0 / np.arange(1, G + 1) if skew else np.ones(G))
    e = rng.choice(G, size=(T, k), p=p / p.sum()).astype(np.int32)
    e[rng.random((T, k)) < empty] = -1
    return e


def find(e, G, layout, room=0, stream=None):
    T, k = e.shape
    sizes = torch.full((G,), -5, dtype=torch.int32, device="cuda")
    rows = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
    m = torch.full((max(room, 1),), -5, dtype=torch.int32, device="cuda")
    x = torch.from_numpy(e).cuda() if T else None
    if layout == "ragged":
        dg.expert_rows_ragged(x, sizes, rows, T, k, G, stream=stream)
    elif layout == "masked":
        dg.expert_rows_masked(x, sizes, rows, T, k, G, room, stream=stream)
    else:
        dg.expert_rows_contiguous(x, sizes, rows, m, T, k, G, room, stream=stream)
    torch.cuda.synchronize()
    return sizes.cpu().numpy(), rows.cpu().numpy(), m[:room].cpu().numpy()


SHAPES = [(1, 1, 1), (1, 8, 2), (7, 3, 8), (61, 8, 2), (500, 1024, 32), (1000, 17, 1), (2049, 60, 6),
          (4096, 256, 8), (9001, 5, 3)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("layout", ["ragged", "contiguous", "masked"])
@pytest.mark.parametrize("skew", [False, True])
def test_rows(shape, layout, skew):
    T, G, k = shape
    e = choices(T, G, k, seed=T, skew=skew)
    room = {"ragged": 0, "contiguous": (T * k // 128 + G + 1) * 128, "masked": max(1, T * k)}[layout]
    if layout == "masked" and G * room >= 2 ** 31:
        pytest.skip("more rows than an index holds")
    got, want = find(e, G, layout, room), M.rows(e, G, layout, room)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    if layout == "contiguous":
        assert np.array_equal(got[2], want[2])


@pytest.mark.parametrize("G", [1021, 1022, 1023, 1024])
@pytest.mark.parametrize("layout", ["ragged", "contiguous", "masked"])
def test_most_experts_and_few_choices(G, layout):
    e = choices(9, G, 4, seed=G)
    e[0, 0], e[1, 1] = G - 1, 0
    room = {"ragged": 0, "contiguous": 37 * 128, "masked": 36}[layout]
    got, want = find(e, G, layout, room), M.rows(e, G, layout, room)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    if layout == "contiguous":
        assert np.array_equal(got[2], want[2])


@pytest.mark.parametrize("T,G,k", [(33000, 64, 8), (70001, 1024, 2), (300000, 256, 1)])
def test_many_rows(T, G, k):
    e = choices(T, G, k, seed=3, skew=True)
    sizes, rows, _ = find(e, G, "ragged")
    flat = e.flatten()
    on = flat >= 0
    order = np.argsort(flat[on], kind="stable")
    want = np.full(flat.shape, -1, np.int32)
    want[np.flatnonzero(on)[order]] = np.arange(on.sum())
    assert np.array_equal(rows.flatten(), want)
    assert np.array_equal(sizes, np.bincount(flat[on], minlength=G))


@pytest.mark.parametrize("layout", ["ragged", "contiguous", "masked"])
def test_no_tokens_and_no_choices(layout):
    for T in (0, 5):
        e = np.full((T, 2), -1, np.int32)
        sizes, rows, m = find(e, 4, layout, 256)
        assert (sizes == 0).all() and (rows == -1).all()
        assert layout != "contiguous" or (m == -1).all()


def test_experts_out_of_range_are_reported():
    e = choices(100, 6, 2, seed=1)
    bad = e.copy()
    bad[3, 0], bad[50, 1], bad[99, 1] = 6, -2, 2 ** 31 - 1
    clean = np.where((bad < 0) | (bad >= 6), -1, bad).astype(np.int32)
    for layout, room in (("ragged", 0), ("contiguous", 1024), ("masked", 200)):
        got = find(bad, 6, layout, room)
        assert dg.get_device_status() == 9
        want = M.rows(clean, 6, layout, room)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


# (72 choices an expert on average, below 128: three segments of 128 rows hold them)
@pytest.mark.parametrize("layout,room,code", [("masked", 9, 8), ("contiguous", 384, 0), ("contiguous", 256, 10),
                                              ("contiguous", 0, 10), ("masked", 0, 8)])
def test_choices_without_room(layout, room, code):
    e = choices(120, 3, 2, seed=4)
    got, want = find(e, 3, layout, room), M.rows(e, 3, layout, room)
    assert dg.get_device_status() == code
    assert all(np.array_equal(a, b) for a, b in zip(got[:2], want[:2]))
    if layout == "contiguous":
        assert np.array_equal(got[2], want[2])


# ---------------------------------------------------------------- dispatch ----
def normal(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)


@pytest.mark.parametrize("T,K,G,k", [(1, 8, 4, 1), (7, 7168, 8, 2), (130, 264, 5, 8), (65, 2056, 3, 32),
                                     (300, 1024, 64, 4)])
def test_dispatch_bf16(T, K, G, k):
    e = choices(T, G, k, seed=K)
    _, rows, _ = M.rows(e, G, "ragged")
    X, D = normal(T, K, seed=1), torch.full((T * k, K), KEEP, dtype=BF16, device="cuda")
    dg.dispatch_rows_bf16(X, torch.from_numpy(rows).cuda(), D, T, K, k, T * k)
    want = torch.full_like(D, KEEP)
    for j in range(k):
        on = rows[:, j] >= 0
        want[torch.from_numpy(rows[on, j]).long().cuda()] = X[torch.from_numpy(on).cuda()]
    assert torch.equal(D, want)


@pytest.mark.parametrize("T,K,G,k,layout", [(1, 128, 4, 1, "masked"), (61, 7168, 8, 2, "masked"),
                                            (33, 640, 3, 8, "masked"), (300, 1152, 5, 4, "contiguous"),
                                            (257, 512, 40, 6, "contiguous")])
@pytest.mark.parametrize("ue8m0", [False, True])
def test_dispatch_fp8(T, K, G, k, layout, ue8m0):
    e = choices(T, G, k, seed=K)
    max_m = T * k + 3 if layout == "masked" else (T * k // 128 + G) * 128
    groups = G if layout == "masked" else 1
    _, rows, _ = M.rows(e, G, layout, max_m)
    kb = (K + 511) // 512 if ue8m0 else K // 128
    ld, ld_out = (T + 3) // 4 * 4 + 4, (max_m + 3) // 4 * 4
    g = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randint(0, 256, (T, K), generator=g, device="cuda", dtype=torch.uint8)
    sa = torch.randint(1, 2 ** 30, (kb, ld), generator=g, device="cuda", dtype=torch.int32)
    A = torch.full((groups, max_m, K), 99, dtype=torch.uint8, device="cuda")
    out = torch.full((groups, kb, ld_out), -9, dtype=torch.int32, device="cuda")
    want, want_sa = A.clone(), out.clone()
    r = torch.from_numpy(rows).cuda()
    if ue8m0:
        dg.dispatch_rows_fp8_1x128_ue8m0(Q, sa, ld, r, A, out, ld_out, T, K, k, groups, max_m)
    else:
        dg.dispatch_rows_fp8_1x128(Q, sa.view(torch.float32), ld, r, A, out.view(torch.float32), ld_out, T, K,
                                   k, groups, max_m)
    for t in range(T):
        for j in range(k):
            if rows[t, j] >= 0:
                z, m = divmod(int(rows[t, j]), max_m)
                want[z, m] = Q[t]
                want_sa[z, :, m] = sa[:, t]
    assert torch.equal(A, want) and torch.equal(out, want_sa)


def test_rows_out_of_range_are_left_out():
    T, K = 9, 256
    rows = torch.tensor([[0], [5], [-1], [6], [2 ** 31 - 1], [-2], [1], [2], [3]], dtype=torch.int32).cuda()
    X, D = normal(T, K), torch.full((8, K), KEEP, dtype=BF16, device="cuda")
    dg.dispatch_rows_bf16(X, rows, D, T, K, 1, 6)
    assert dg.get_device_status() == 9
    want = torch.full_like(D, KEEP)
    for t, r in enumerate(rows.flatten().tolist()):
        if 0 <= r < 6:
            want[r] = X[t]
    assert torch.equal(D, want)
    Y, out = normal(8, K, seed=2), torch.full((T, K), KEEP, dtype=BF16, device="cuda")
    dg.combine_rows(Y, rows, None, X, out, T, K, 1, 6)
    assert dg.get_device_status() == 9
    ok = torch.tensor([0 <= r < 6 for r in rows.flatten().tolist()]).cuda()
    assert torch.equal(out[~ok], X[~ok])
    dY, dw = torch.full_like(D, KEEP), torch.full((T, 1), KEEP, device="cuda")
    dg.combine_rows_backward(X, Y, rows, None, dY, dw, T, K, 1, 6)
    assert dg.get_device_status() == 9
    assert torch.equal(dY, want) and (dw[~ok] == 0).all()


# ----------------------------------------------------------------- combine ----
SUMS = [(1, 8, 4, 1), (7, 7168, 8, 2), (130, 264, 5, 8), (65, 2056, 3, 32), (300, 1024, 64, 4), (3, 512, 9, 9)]


@pytest.mark.parametrize("T,K,G,k", SUMS)
@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False), (True, False), (False, True)])
def test_combine(T, K, G, k, weighted, residual):
    e = choices(T, G, k, seed=K)
    e[0] = -1    # a token without a row
    _, rows, _ = M.rows(e, G, "ragged")
    Y, res = normal(T * k, K, seed=1), normal(T, K, seed=2, scale=2.0) if residual else None
    w = torch.rand(T, k, device="cuda") if weighted else None
    out = torch.full((T, K), KEEP, dtype=BF16, device="cuda")
    r = torch.from_numpy(rows).cuda()
    dg.combine_rows(Y, r, w, res, out, T, K, k, T * k)
    want, mag = M.combine(Y.float().cpu().numpy(), rows, None if w is None else w.cpu().numpy(),
                          None if res is None else res.float().cpu().numpy())
    R.check_close(out.cpu(), torch.from_numpy(want), (k + 1) * U * torch.from_numpy(mag), "combine")
    if residual:   # in place
        dg.combine_rows(Y, r, w, res, res, T, K, k, T * k)
        assert torch.equal(res, out)


def test_combine_ignores_rows_that_no_choice_names():
    # rows that hold infinities or NaN reach only the tokens that name them
    Y = normal(6, 256)
    Y[1], Y[3] = float("inf"), float("nan")
    rows = torch.tensor([[0, 2], [-1, 4], [5, -1], [-1, -1], [1, 0], [3, -1]], dtype=torch.int32).cuda()
    w = torch.tensor([[1.0, 2], [float("nan"), 1], [1, float("inf")], [float("nan")] * 2, [0.5, 1], [0, 0]]).cuda()
    out = torch.empty(6, 256, dtype=BF16, device="cuda")
    dg.combine_rows(Y, rows, w, None, out, 6, 256, 2, 6)
    assert torch.isfinite(out[:3]).all() and (out[3] == 0).all()
    assert torch.isinf(out[4]).all() and torch.isnan(out[5]).all()
    assert torch.equal(out[1], Y[4]) and torch.equal(out[2], Y[5])


@pytest.mark.parametrize("T,K,G,k", SUMS)
@pytest.mark.parametrize("weighted", [True, False])
def test_combine_gradient(T, K, G, k, weighted):
    e = choices(T, G, k, seed=K)
    _, rows, _ = M.rows(e, G, "ragged")
    Y, dO = normal(T * k, K, seed=1), normal(T, K, seed=2, scale=0.02)
    w = torch.rand(T, k, device="cuda") if weighted else None
    r = torch.from_numpy(rows).cuda()
    dY, dw = torch.full_like(Y, KEEP), torch.full((T, k), KEEP, device="cuda")
    dg.combine_rows_backward(dO, Y, r, w, dY, dw, T, K, k, T * k)
    alone = torch.full_like(Y, KEEP)
    dg.combine_rows_backward(dO, None, r, w, alone, None, T, K, k, T * k)
    assert torch.equal(dY, alone)
    wants, named = torch.full(Y.shape, KEEP, dtype=torch.float64), torch.zeros(T * k, dtype=torch.bool)
    Yc, dc = Y.double().cpu(), dO.double().cpu()
    for t in range(T):
        for j in range(k):
            x = int(rows[t, j])
            if x < 0:
                assert dw[t, j] == 0
                continue
            named[x] = True
            wants[x] = dc[t] * (float(w[t, j]) if weighted else 1.0)
            p = dc[t] * Yc[x]
            assert abs(float(dw[t, j]) - float(p.sum())) <= (K / 8 + 16) * U * float(p.abs().sum())
    assert (dY.cpu()[~named] == KEEP).all()
    R.check_close(dY.cpu()[named], wants[named], 2 * U * wants[named].abs(), "gradient of the rows")


def test_dispatch_and_its_gradient_are_each_others_transpose():
    # <D(x), y> = <x, D^T(y)> in whole numbers
    T, K, G, k = 50, 264, 6, 3
    _, rows, _ = M.rows(choices(T, G, k, seed=8), G, "ragged")
    r = torch.from_numpy(rows).cuda()
    x = torch.randint(-4, 5, (T, K), device="cuda").to(BF16)
    y = torch.randint(-4, 5, (T * k, K), device="cuda").to(BF16)
    D, back = torch.zeros(T * k, K, dtype=BF16, device="cuda"), torch.empty(T, K, dtype=BF16, device="cuda")
    dg.dispatch_rows_bf16(x, r, D, T, K, k, T * k)
    dg.combine_rows(y, r, None, None, back, T, K, k, T * k)
    assert (D.double() * y.double()).sum() == (x.double() * back.double()).sum()


def test_streams_graphs_and_limits():
    T, K, G, k = 700, 1024, 16, 4
    e = torch.from_numpy(choices(T, G, k, seed=5)).cuda()
    sizes, rows = torch.empty(G, dtype=torch.int32, device="cuda"), torch.empty(T, k, dtype=torch.int32, device="cuda")
    X, w, dO = normal(T, K), torch.rand(T, k, device="cuda"), normal(T, K, seed=3)
    D, out = torch.zeros(T * k, K, dtype=BF16, device="cuda"), torch.zeros(T, K, dtype=BF16, device="cuda")
    dY, dw = torch.zeros_like(D), torch.zeros(T, k, device="cuda")
    outs = (sizes, rows, D, out, dY, dw)

    def chain(stream=None):
        dg.expert_rows_ragged(e, sizes, rows, T, k, G, stream=stream)
        dg.dispatch_rows_bf16(X, rows, D, T, K, k, T * k, stream=stream)
        dg.combine_rows(D, rows, w, X, out, T, K, k, T * k, stream=stream)
        dg.combine_rows_backward(dO, D, rows, w, dY, dw, T, K, k, T * k, stream=stream)

    def again(run):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))

    chain()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    again(lambda: chain(side))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        chain()
    again(g.replay)
    for sms in (1, 3, 132):
        dg.set_num_sms(sms)
        try:
            grids = launched(chain)
            again(chain)
        finally:
            dg.set_num_sms(0)
        assert len(grids) == 4 and all(b <= sms for b, _, _ in grids)
    # a sort of more than one block under a limit
    big = torch.from_numpy(choices(40000, 32, 2, seed=1)).cuda()
    n, at = torch.empty(32, dtype=torch.int32, device="cuda"), torch.empty(40000, 2, dtype=torch.int32, device="cuda")
    call = lambda s=None: dg.expert_rows_ragged(big, n, at, 40000, 2, 32, stream=s)
    call()
    torch.cuda.synchronize()
    free = at.clone()
    dg.set_num_sms(3)
    try:
        at.zero_()
        call()
        assert all(b <= 3 for b, _, _ in launched(call))
        torch.cuda.synchronize()
    finally:
        dg.set_num_sms(0)
    assert torch.equal(at, free)


def test_operands_past_32_bits():
    # 4.9e9 elements: rows at both ends, with their scales
    R, K, T = 600000, 8192, 4
    assert R * K > 2 ** 32
    at = torch.tensor([[0, R - 1], [R // 2, 5], [R - 2, 300001], [7, -1]], dtype=torch.int32).cuda()
    X = normal(T, K, seed=1)
    D = torch.zeros(R, K, dtype=BF16, device="cuda")
    dg.dispatch_rows_bf16(X, at, D, T, K, 2, R)
    for t in range(T):
        for r in at[t].tolist():
            if r >= 0:
                assert torch.equal(D[r], X[t])
    assert int((D[:, 0] != 0).sum()) == 7
    out, w = torch.empty(T, K, dtype=BF16, device="cuda"), torch.full((T, 2), 0.5, device="cuda")
    dg.combine_rows(D, at, w, None, out, T, K, 2, R)
    assert torch.equal(out[:3], X[:3]) and torch.equal(out[3], 0.5 * X[3])
    dY, dw = torch.zeros_like(D), torch.empty(T, 2, device="cuda")
    dg.combine_rows_backward(X, D, at, w, dY, dw, T, K, 2, R)
    assert torch.equal(dY[R - 1], 0.5 * X[0]) and torch.equal(dY[300001], 0.5 * X[2])
    assert int((dY[:, 0] != 0).sum()) == 7
    del D, dY
    G, max_m = 64, 10000
    Q = torch.randint(0, 256, (T, K), device="cuda", dtype=torch.uint8)
    sa = torch.rand(K // 128, 4, device="cuda") + 0.5
    A = torch.zeros(G, max_m, K, dtype=torch.uint8, device="cuda")
    out_sa = torch.zeros(G, K // 128, max_m, device="cuda")
    at = torch.tensor([[0, G * max_m - 1], [320000, 5], [G * max_m - 2, 300001], [7, -1]], dtype=torch.int32).cuda()
    dg.dispatch_rows_fp8_1x128(Q, sa, 4, at, A, out_sa, max_m, T, K, 2, G, max_m)
    for t in range(T):
        for r in at[t].tolist():
            if r >= 0:
                z, m = divmod(r, max_m)
                assert torch.equal(A[z, m], Q[t]) and torch.equal(out_sa[z, :, m], sa[:, t])
    assert int((out_sa[:, 0] != 0).sum()) == 7


@pytest.mark.parametrize("team", [(9451, 360, 1), (2000, 2048, 3), (700, 2000, 4), (40, 8, 2), (300, 4096, 9), (5, 16384, 2)],
                         ids=lambda s: "x".join(map(str, s)))
def test_teams_of_the_gradient(team):
    # few and many tokens, short and long rows: each takes teams of another size
    T, K, k = team
    _, rows, _ = M.rows(choices(T, 16, k, seed=T), 16, "ragged")
    Y, dO, w = normal(T * k, K, seed=1), normal(T, K, seed=2), torch.rand(T, k, device="cuda")
    r = torch.from_numpy(rows).cuda()
    dY, dw = torch.full_like(Y, KEEP), torch.full((T, k), KEEP, device="cuda")
    dg.combine_rows_backward(dO, Y, r, w, dY, dw, T, K, k, T * k)
    on = r >= 0
    at = r.clamp_min(0).long()
    prod = dO.double()[:, None] * Y[at].double()
    lim = (K / 8 + 16) * U * prod.abs().sum(2)
    assert ((dw.double() - torch.where(on, prod.sum(2), 0.0)).abs() <= torch.where(on, lim, 0.0)).all()
    want = torch.full(Y.shape, KEEP, dtype=torch.float64, device="cuda")
    want[at[on]] = (dO.double()[:, None] * w.double()[..., None])[on]
    R.check_close(dY, want, 2 * U * want.abs(), "gradient of the rows")
    out = torch.full_like(dO, KEEP)
    dg.combine_rows(Y, r, w, dO, out, T, K, k, T * k)
    sums = torch.where(on[..., None], w.double()[..., None] * Y[at].double(), 0.0)
    R.check_close(out, dO.double() + sums.sum(1), (k + 1) * U * (dO.double().abs() + sums.abs().sum(1)), "combine")
