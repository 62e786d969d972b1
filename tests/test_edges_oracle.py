"""The plain 64-bit forms that the GPU tests of the sub-layer edge operators
compare against: gradients against central differences of the forward, and
properties that the definitions fix.  No GPU."""
import numpy as np
import pytest

from tests import _edges as O


def differences(f, x, d=1e-6):
    g = np.zeros_like(x)
    it = np.nditer(x, flags=["multi_index"])
    for _ in it:
        i = it.multi_index
        keep = x[i]
        x[i] = keep + d
        up = f()
        x[i] = keep - d
        g[i] = (up - f()) / (2 * d)
        x[i] = keep
    return g


@pytest.mark.parametrize("D,R,inter", [(8, 8, False), (8, 4, True), (7, 4, False), (6, 0, False)])
def test_qk_gradient_is_the_difference_quotient(D, R, inter):
    r = np.random.default_rng(D + R)
    x, dy, gamma = r.normal(size=(3, 2, D)), r.normal(size=(3, 2, D)), r.normal(size=D)
    cos, sin = (t[[5, 0, 9]].astype(float) for t in O.rope_table(10, R))
    f = lambda: (dy * O.qk_fwd(x, gamma, cos, sin, R, inter, 1e-3)[0]).sum()  # noqa: E731
    dx, _, dg, _ = O.qk_bwd(dy, x, gamma, cos, sin, R, inter, 1e-3)
    # central differences of step 1e-6: 1e-12 of curvature, 1e-16 / 1e-6 of rounding
    assert np.allclose(dx, differences(f, x), atol=1e-7)
    assert np.allclose(dg, differences(f, gamma), atol=1e-7)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_is_the_difference_quotient(score, renorm):
    r = np.random.default_rng(1)
    l, dw = r.normal(size=(4, 9)), r.normal(size=(4, 3))
    ids = O.top(l, 3)
    ids[1, 2] = -1
    f = lambda: (2.5 * dw * O.router_scores(l, ids, score, renorm)).sum()  # noqa: E731
    d, _ = O.router_bwd(dw, l, ids, score, renorm, 2.5)
    assert np.allclose(d, differences(f, l), atol=1e-7)


def test_combine_gradient_is_the_difference_quotient():
    r = np.random.default_rng(2)
    ids = np.array([[0, 2], [2, -1], [1, 2], [-1, -1]])
    _, off, row, slot = O.sort(ids, 3, 4, 4 * 2 + 3 * 3)
    ys, w, df = r.normal(size=(len(slot), 5)), r.normal(size=(4, 2)), r.normal(size=(4, 5))
    f = lambda: (df * O.combine(ys, w, row)[0]).sum()  # noqa: E731
    dys, dw, _ = O.combine_bwd(df, ys, w, row, slot)
    assert np.allclose(dys, differences(f, ys), atol=1e-7)
    assert np.allclose(dw, differences(f, w), atol=1e-7)
    # the gradient of dispatch is the unweighted combine
    x = r.normal(size=(4, 5))
    g = lambda: (ys * O.dispatch(x, slot, 2)).sum()  # noqa: E731
    assert np.allclose(O.combine(ys, None, row)[0], differences(g, x), atol=1e-7)


def test_rotation_keeps_norms_and_turns_by_differences_of_position():
    r = np.random.default_rng(3)
    x, y = r.normal(size=(1, 1, 16)), r.normal(size=(1, 1, 16))
    a = np.arange(64)[:, None] * 100.0 ** (-np.arange(8) / 8)
    at = lambda v, p: O.turn(v, np.cos(a[[p]]), np.sin(a[[p]]), 16, False)  # noqa: E731
    assert np.isclose((at(x, 40) * at(y, 33)).sum(), (at(x, 10) * at(y, 3)).sum())
    assert np.isclose((at(x, 40) ** 2).sum(), (x ** 2).sum())


def test_sort_is_a_stable_permutation_with_padding():
    r = np.random.default_rng(4)
    ids = r.integers(-1, 5, size=(40, 3))
    counts, off, row, slot = O.sort(ids, 5, 8, 40 * 3 + 5 * 7)
    assert counts.sum() == (ids >= 0).sum() and np.all(np.diff(off) % 8 == 0)
    kept = row.reshape(-1)[ids.reshape(-1) >= 0]
    assert len(set(kept.tolist())) == len(kept) and np.array_equal(slot[kept],
                                                                   np.flatnonzero(ids.reshape(-1) >= 0))
    for e in range(5):
        seg = slot[off[e]:off[e + 1]]
        real = seg[:counts[e]]
        assert np.all(np.diff(real) > 0) and np.all(ids.reshape(-1)[real] == e)
        assert np.all(seg[counts[e]:] == -1)
    assert np.all(slot[off[-1]:] == -1)
