"""The comparison of the prompt attention's moving maxima can fail (CPU): an online softmax with
a mistake in its rescaling, computed in 64 bits, leaves the tolerance; one without does not."""
import numpy as np
import pytest

from tests.test_prefill_edges_gpu import staircase

BLOCK, LIFT, MOST = 128, 7.0, 15.0


def online(y, V, mistake=None):
    """Softmax of the rows of y (log2) over blocks of keys, the unit moved as the kernel moves it."""
    n, keys = y.shape
    m = l = o = None
    for k in range(0, keys, BLOCK):
        x = y[:, k:k + BLOCK]
        top = x.max(1)
        if k == 0:
            m, l, o = top - LIFT, np.zeros(n), np.zeros((n, V.shape[1]))
        else:
            new = np.where(top > m + MOST, top - LIFT, m)
            f = np.exp2(m - new)
            m = new
            fo = np.roll(f, -8) if mistake == "rows" else f
            fl = np.ones(n) if mistake == "sum" else f
            fo = np.ones(n) if mistake == "output" else fo
            late = mistake == "late"            # this block's weights are rescaled as well
            l, o = l * fl, o * fo[:, None]
            if mistake == "columns":
                o[:, ::2] *= np.where(f < 1, 0.5, 1.0)[:, None]
        p = np.exp2(x - m[:, None])
        if k and late:
            p = p * np.where(f < 1, 0.96, 1.0)[:, None]
        l, o = l + p.sum(1), o + p @ V[k:k + BLOCK]
    return o / l[:, None]


@pytest.mark.parametrize("mistake", [None, "rows", "sum", "output", "late", "columns"])
def test_mistakes_in_the_rescaling_show(mistake):
    _, y, V, ref, tol = staircase(1)
    inside = (np.abs(online(y, V, mistake) - ref) <= tol).all()
    assert inside == (mistake is None)


def test_tolerance_is_tight_where_the_weight_is():
    _, _, _, ref, tol = staircase(1)
    near = ref > 2.0 ** -14
    assert (tol[near] <= 0.01 * ref[near]).all() and near.sum(1).min() >= 1
    assert near.sum() >= 1.5 * len(ref)
