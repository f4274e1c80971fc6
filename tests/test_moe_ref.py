"""The definitions that the expert layer's operators are tested against, on their
own: gradients against differences, rows against what a layout has to hold."""
import numpy as np
import pytest

from tests import moe_ref as M


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(sigmoid, renorm):
    rng = np.random.default_rng(3)
    x, dw = rng.normal(size=(5, 12)), rng.normal(size=(5, 4))
    e, w = M.route(x, None, 4, sigmoid, renorm=renorm, scale=1.7)

    def value(x):
        s = np.stack([M.scores(r, sigmoid)[0] for r in x])
        v = np.take_along_axis(s, e.astype(np.int64), 1)
        if renorm:
            v = v / (v.sum(1, keepdims=True) + (1e-20 if sigmoid else 0.0))
        return 1.7 * (v * dw).sum()

    assert np.allclose(value(x), (w * dw).sum())
    got, mag = M.route_backward(x, e, dw, sigmoid, renorm, 1.7)
    assert (np.abs(got) <= mag + 1e-15).all()
    for t in range(5):
        for i in range(12):
            h = np.zeros_like(x)
            h[t, i] = 1e-6
            assert abs((value(x + h) - value(x - h)) / 2e-6 - got[t, i]) < 1e-8


def test_choice():
    x = np.array([[0.0, 2.0, 2.0, -np.inf, np.nan, 1.0, -1.0, 3.0]])
    assert M.route(x, None, 4, True)[0].tolist() == [[7, 1, 2, 5]]
    # groups of two, by the best one of each: values of 2, 2, 1, 3, the first two equal
    e, w = M.route(x, None, 3, True, 4, 2, 1)
    assert e.tolist() == [[7, 1, 0]] and abs(w.sum() - 1.0) < 1e-12
    none = np.full((1, 4), -np.inf)
    e, w = M.route(none, None, 2, False)
    assert e.tolist() == [[-1, -1]] and (w == 0).all()


@pytest.mark.parametrize("layout,room", [("ragged", 0), ("contiguous", 512), ("masked", 16)])
def test_rows(layout, room):
    rng = np.random.default_rng(1)
    e = rng.integers(-1, 3, size=(14, 2)).astype(np.int32)
    sizes, rows, m = M.rows(e, 3, layout, room)
    used = rows[rows >= 0]
    assert len(set(used.tolist())) == len(used) == (e >= 0).sum() == sizes.sum()
    if layout == "contiguous":
        assert (m[rows[e >= 0]] == e[e >= 0]).all() and (m >= 0).sum() == len(used)
