"""The 64-bit form of the router's gradient with dropped slots: the difference
quotient of the forward's weights over the whole choice.  No GPU."""
import numpy as np
import pytest

from tests import _edges as O
from tests.test_edges_oracle import differences


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_dropped_slots_keep_their_share_of_the_sum(score, renorm):
    r = np.random.default_rng(5)
    l, dw = r.normal(size=(5, 9)), r.normal(size=(5, 3))
    ids = O.top(l, 3)
    kept = ids.copy()
    kept[1, 2] = kept[2, 0] = kept[3, 0] = kept[3, 1] = -1
    kept[4] = -1
    dw_kept = np.where(kept >= 0, dw, 0)
    f = lambda: (2.5 * dw_kept * O.router_scores(l, ids, score, renorm)).sum()  # noqa: E731
    want = differences(f, l)
    assert np.allclose(O.router_bwd(dw_kept, l, ids, score, renorm, 2.5)[0], want, atol=1e-7)
    assert np.allclose(O.router_bwd(dw, l, kept, score, renorm, 2.5)[0], want, atol=1e-7)
    # the weights of the slots that were kept are the forward's
    w = O.router_scores(l, ids, score, renorm)
    assert np.array_equal(O.router_scores(l, kept, score, renorm), np.where(kept >= 0, w, 0))


def test_one_row_worked_by_hand():
    """Two equal logits chosen, one slot dropped, dw = (1, 0): w = (1/2, 1/2),
    so the gradient is w_0 w_1 = 1/4 and its negative."""
    d, _ = O.router_bwd(np.array([[1.0, 0]]), np.array([[2.0, 2, -3]]), np.array([[0, -1]]),
                        "softmax", True, 1.0)
    assert np.allclose(d, [[0.25, -0.25, 0]])
