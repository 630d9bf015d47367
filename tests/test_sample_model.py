"""The rule of sampled acceptance, on CPU: whatever the drafter proposes, the emitted token
is distributed as the target; and the page pool's model keeps its counts."""
import numpy as np
import pytest

from tests import serving_model as sm


def emitted(w, children, g):
    """The distribution of a node's emitted token: every test's chance, then the draw."""
    out, reach = np.zeros(len(w)), 1.0
    left = np.array(w, np.float64)
    for x, limit, rest in sm.accept_steps(w, children, g):
        a = min(1.0, limit)
        out[x] += reach * a
        reach *= 1.0 - a
        left = rest
        if left.sum() == 0:
            return out
    return out + reach * left / left.sum()


@pytest.mark.parametrize("seed", range(5))
def test_chosen_candidates_leave_the_target_unchanged(seed):
    r = np.random.default_rng(seed)
    p = r.dirichlet(np.ones(7))
    for n in range(8):
        got = emitted(p, r.permutation(7)[:n], None)
        assert np.allclose(got, p, atol=1e-14)


@pytest.mark.parametrize("seed", range(5))
def test_drawn_candidates_leave_the_target_unchanged(seed):
    """Averaged over every draw without replacement of two children from g."""
    r = np.random.default_rng(seed)
    V = 5
    p, g = r.dirichlet(np.ones(V)), r.dirichlet(np.ones(V))
    got = np.zeros(V)
    for a in range(V):
        for b in range(V):
            if a != b:
                got += g[a] * g[b] / (1 - g[a]) * emitted(p, [a, b], g)
    assert np.allclose(got, p, atol=1e-14)


def test_pool_model_keeps_its_counts():
    r = np.random.default_rng(1)
    pool = sm.Pool(6, 12, 80, 4)
    length = np.zeros(6, np.int64)
    for step in range(60):
        new = np.minimum(length + r.integers(0, 6, 6), 44)
        assert pool.reserve(length, new) is not None
        length = new
        pool.check()
        r0 = int(r.integers(0, 6))
        keep = np.full(6, -1)
        keep[r0] = 0
        pool.release(keep)
        length[r0] = 0
        src = np.full(6, -1)
        src[r0] = (r0 + 1) % 6
        length[r0] = length[src[r0]]
        pool.fork(src, length)
        pool.check()
        pool.compact()
        pool.check()
