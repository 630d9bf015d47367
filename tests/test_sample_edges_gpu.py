"""GPU tests of tv_tree_sample at uniform numbers next to the boundaries they are compared with.

Floats decide a test or a draw only where a bound on their error (about 5e-6) allows it.  The
numbers here are floats next to a boundary, most of them within 2^-25 of it, so that nothing
but the exact sums can tell which side they lie on.  A number is left out where the exact sums
need not tell either: weights are held to 2^-37 of themselves and half a unit, 2^-45 of the
row's largest, so that a boundary moves by less than 2^-30 here (at most 2^-27 of the row's sum
if every one of 2^18 roundings went the same way; they are independent, 2^9 of them count)."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import serving_model as sm
from tests.test_sample_gpu import call, make

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
FAR = 2.0 ** -30


def beside(x, side, far=FAR):
    """The float in [0, 1) next to x from below (side 0) or above, at least `far` away."""
    aim = x + far if side else x - far
    f = np.float32(aim)
    if f < aim if side else f > aim:
        f = np.nextafter(f, np.float32(2 * side - 1), dtype=np.float32)
    return float(f) if 0 <= f < 1 else None


def compare(s, **kw):
    B = len(s["uniforms"])
    got, status = call(s, **kw)
    assert status == 0
    x = s["logits"].double().numpy()
    for b in range(B):
        want = sm.sample_tree(x[b], s["parent"][b].numpy(), s["tokens"][b].numpy(),
                              s["uniforms"][b].numpy(), float(s["temperature"][b]),
                              None if s["draft"] is None else s["draft"][b].double().numpy())
        assert got[0][b] == want[0] and np.array_equal(got[2][b], want[2]), b


def draws(x, T, seed, near=None):
    """Inputs whose only work is a draw next to a boundary of the row's running sum, or up to
    2^near away from it."""
    B, V = x.shape
    r = np.random.default_rng(seed)
    u = np.zeros((B, 1), np.float32)
    for b in range(B):
        w = sm.weights(x[b].double().numpy(), T)
        total = np.cumsum(w)
        inner = np.flatnonzero(w[:-1] > 2.0 ** -24 * total[-1])
        # (a token next to the boundary on either side)
        at = r.choice(inner) if len(inner) else 0
        far = FAR if near is None else 2.0 ** r.uniform(-26, near)
        v = beside(total[at] / total[-1], int(r.integers(0, 2)), far)
        u[b, 0] = r.random() if v is None else v
    return dict(logits=x[:, None], parent=torch.full((B, 1), -1, dtype=torch.int32),
                tokens=torch.zeros((B, 1), dtype=torch.int32), uniforms=torch.from_numpy(u),
                temperature=torch.full((B,), float(np.float32(T))), draft=None, by_node=False)


@pytest.mark.parametrize("T", [0.7, 1.0, 1.3])
@pytest.mark.parametrize("B,V,dtype", [(24, 50257, "fp32"), (8, 163840, "bf16"),
                                       (640, 4099, "fp32"), (200, 2048, "bf16")])
def test_draws_next_to_a_boundary(B, V, dtype, T):
    """Clusters of 16 CTAs to 1, a third of the distributions peaked, a third wide."""
    r = np.random.default_rng(B + V)
    spread = np.array([0.5, 2.0, 5.0])[np.arange(B) % 3, None]
    x = torch.from_numpy((r.normal(size=(B, V)) * spread).astype(np.float32))
    compare(draws(x.bfloat16() if dtype == "bf16" else x, float(np.float32(T)), B))


@pytest.mark.parametrize("T", [0.7, 1.3, 0.30103])
@pytest.mark.parametrize("B,V", [(640, 16384), (3, 1 << 18)])
@pytest.mark.parametrize("rise", [1, -1])
def test_slowly_moving_maxima(B, V, T, rise):
    """Weights that climb (or fall) by 2^18 along the row: the running maxima move at every
    step, every value's weight is a product of many exponentials, and the mean exponent is as
    large as it can be.  With 1/T that floats do not hold."""
    ramp = np.linspace(-18, 0, V)[::rise] * np.log(2.0) * T
    r = np.random.default_rng(V)
    x = ramp + 0.01 * r.normal(size=(B, V))
    compare(draws(torch.from_numpy(x.astype(np.float32)), float(np.float32(T)), V))


@pytest.mark.parametrize("draft", [None, "depth"])
@pytest.mark.parametrize("seed", range(4))
def test_tests_and_residual_draws_next_to_a_boundary(draft, seed):
    """Up to three children are refused with numbers well past their limits; then a child is
    tested next to its limit, or the bonus token is drawn next to a boundary of what is left."""
    B, V, Q = 48, 3001, 6
    s = make(50 + seed, B, Q, V, draft=draft, wide=8)
    s["parent"][:, 1:] = 0
    r = np.random.default_rng(60 + seed)
    for b in range(B):
        g = None if draft is None else s["draft"][b, 0].double().numpy()
        # children in the order of a draw without replacement, or the most likely ones
        score = (s["logits"][b, 0].double().numpy() if g is None else np.log(g))
        s["tokens"][b, 1:] = torch.from_numpy(
            np.argsort(-(score + (0 if g is None else r.gumbel(size=V))))[:Q - 1].astype(np.int32))
        T = float(s["temperature"][b])
        w = sm.weights(s["logits"][b, 0].double().numpy(), T)
        u = np.full(Q, 1 - 2.0 ** -24, np.float32)
        u[0] = r.random()
        refuse = int(r.integers(0, 4))
        left = w
        for i, (_, limit, rest) in enumerate(sm.accept_steps(w, s["tokens"][b, 1:].tolist(), g)):
            if limit >= 0.999 or rest.sum() < 0.01 * w.sum():
                u[1 + i] = 0.5 * min(limit, 1.0)     # accepted: the walk goes on with row 1 + i
                break
            if i == refuse:
                # the token's weight is held to 2^-44: of a small one that is a larger share
                far = max(FAR, limit * 2.0 ** -40 / max(left[s["tokens"][b, 1 + i]], 1e-30))
                v = beside(limit, int(r.integers(0, 2)), far)
                u[1 + i] = 0.999 if v is None else v
            left = rest
        else:
            total = np.cumsum(left)
            inner = np.flatnonzero(left[:-1] > 2.0 ** -20 * total[-1])
            v = beside(total[r.choice(inner)] / total[-1], int(r.integers(0, 2)))
            u[0] = u[0] if v is None else v
        s["uniforms"][b] = torch.from_numpy(u)
    compare(s)


@pytest.mark.parametrize("T", [0.7, 1.3, 0.30103])
@pytest.mark.parametrize("rise", [1, -1, 0])
def test_draws_at_any_distance_from_a_boundary(T, rise):
    """2^-26 to 2^-16: where floats leave off and the exact sums take over."""
    B, V = 640, 8192
    r = np.random.default_rng(70 + rise)
    x = 2.0 * r.normal(size=(B, V))
    if rise:
        x = 0.005 * x + np.linspace(-15, 0, V)[::rise] * np.log(2.0) * T
    compare(draws(torch.from_numpy(x.astype(np.float32)), float(np.float32(T)), V, near=-16))


def test_greedy_rows_need_no_drafter():
    """At temperature 0 the drafter's rows are not read: a depth without one is no error, and
    what the rows hold does not matter."""
    s = make(80, 4, 6, 50, draft="depth", wide=1)
    s["temperature"][:] = 0.0
    top = s["logits"].float().argmax(-1).to(torch.int32)
    s["tokens"][:, 1:] = top[:, :-1]                # the whole chain is the target's own
    s["draft"] = torch.full((4, 1, 50), float("nan"))
    got, status = call(s)
    assert status == 0 and (got[0] == 5).all()
    assert np.array_equal(got[2], top.numpy())
    s["temperature"][1] = 1.0                       # a sampled row of the batch does need one
    s["draft"] = torch.full((4, 1, 50), 1.0 / 50)
    s["uniforms"][:, 1] = 0.0
    got, status = call(s)
    assert status == tv.TV_ERR_BOUNDS and got[0].tolist() == [5, 1, 5, 5]


@pytest.mark.parametrize("mass", [0.9, 0.999])
def test_masked_children_are_never_taken(mass):
    """The target allows one token, of which the drafter is nearly sure, and the children are
    others: every rejection leaves a tenth (or a thousandth) of the weight, down to less than the
    exact sums hold, and the allowed token has to be drawn all the same."""
    B, V, Q = 4, 64, 24
    r = np.random.default_rng(90)
    s = make(90, B, Q, V, draft="depth")
    s["parent"][:, 1:] = 0
    s["logits"][:, 0] = float("-inf")
    s["draft"] = torch.full((B, Q, V), (1 - mass) / (V - 1))
    for b in range(B):
        order = r.permutation(V).astype(np.int32)
        s["logits"][b, 0, int(order[0])] = 1.5
        s["draft"][b, :, int(order[0])] = mass
        s["tokens"][b, 1:] = torch.from_numpy(order[1:Q])
    compare(s)
    got, _ = call(s)
    assert (got[0] == 0).all() and (got[2][:, 0] == s["logits"][:, 0].argmax(-1).numpy()).all()
