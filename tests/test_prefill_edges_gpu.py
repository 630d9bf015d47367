"""GPU tests of tv_prefill_attn where it can go wrong: bounds at the ends of their range, NaN
in cut items, weights far below a row's largest, running maxima that move.

The roundings that the tolerances count are those of tests/test_prefill_attn_gpu.py."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_prefill_attn_gpu as base

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("where", [0, 1])
def test_a_prefix_at_the_end_of_the_integers(where):
    """Host bounds without a limit and a prefix of nearly 2^31 keys: the sequence has more
    blocks of keys than were announced, so it and those behind it are left out."""
    s = base.make(31, 1, [40, 40], [5, 5], DL=64, paged=False)
    good = base.run(s)
    s["prefixes"][where] = INT_MAX - 40
    d = base.device(s)
    base.launch(s, d, max_kv_len=INT_MAX, total_kv=90, kv_stride_b=INT_MAX)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == tv.TV_ERR_BOUNDS
    out = d["out"].double().cpu().numpy()
    done = 40 * where
    assert np.array_equal(out[:done], good[:done]) and (out[done:] == -77).all()


def output(s):
    d = base.device(s)
    base.launch(s, d)
    torch.cuda.synchronize()
    return d["out"].double().cpu().numpy()


@pytest.mark.parametrize("H,lens,prefixes", [
    (1, [200], [1500]),      # cut along the keys: a dozen pieces
    (80, [200, 40], [600, 3]),  # whole items
])
def test_a_nan_reaches_the_rows_that_see_it_and_no_other(H, lens, prefixes):
    """Cut or whole, a NaN score makes the row NaN; the other rows keep their bits."""
    s = base.make(32, H, lens, prefixes, DL=64)
    good = output(s)
    q = s["q_nope"].clone()
    s["q_nope"][7, 0, 3] = float("nan")
    out = output(s)
    assert np.isnan(out[7, 0]).all()
    out[7, 0] = good[7, 0]
    assert np.array_equal(out, good)
    s["q_nope"] = q
    for key in (0, 130, prefixes[0] + 50):      # a rope key: of the first piece, another, the last
        k = s["k_pe"].clone()
        s["k_pe"][s["rows"][0][key]] = float("nan")
        out = output(s)
        first = max(0, key - prefixes[0])        # the first query of the sequence that sees it
        assert np.isnan(out[first:lens[0]]).all()
        out[first:lens[0]] = good[first:lens[0]]
        assert np.array_equal(out, good)
        s["k_pe"] = k


def test_values_that_are_nan_are_reported():
    """From the weights: the scores do not show it.  From a key's row: they do as well."""
    s = base.make(33, 2, [90], [40], DL=64)
    good = output(s)
    w = s["w_kv"].clone()
    s["w_kv"][1, 128 + 5, 7] = float("nan")
    out = base.run(s, tv.TV_ERR_BOUNDS)
    assert np.array_equal(out[:, 0], good[:, 0])
    s["w_kv"] = w
    s["c_kv"][s["rows"][0][50], 3] = float("nan")
    out = base.run(s, tv.TV_ERR_BOUNDS)
    assert np.array_equal(out[:10], good[:10]) and np.isnan(out[10:]).all()


def exact_scores(H, x, v, prefix, extra=0):
    """A batch of one query row whose scores are x[j] exactly, in units of log2, and whose
    values are v[j] in the first of 56 columns: keys 0 .. prefix + extra are one latent column,
    values others, both taken over by weights of zeros and ones.  x and v are bf16 numbers."""
    s = base.make(34, H, [1 + extra], [prefix], DL=64)
    for k in ("q_nope", "q_pe", "w_kv"):
        s[k].zero_()
    s["q_nope"][:, :, 0] = 1.0
    s["w_kv"][:, 0, 0] = 1.0
    for d in range(56):
        s["w_kv"][:, 128 + d, 8 + d] = 1.0
    at = s["rows"][0]
    s["c_kv"][at] = 0.0
    s["k_pe"][at] = 0.0
    s["c_kv"][at, 0] = torch.from_numpy(x).bfloat16()
    s["c_kv"][at, 8] = torch.from_numpy(v).bfloat16()
    assert np.array_equal(s["c_kv"][at, 0].double().numpy(), x)
    assert np.array_equal(s["c_kv"][at, 8].double().numpy(), v)
    s["scale"] = float(np.float32(np.log(2.0)))
    return s


@pytest.mark.parametrize("H", [1, 160])     # cut along the keys, whole items
@pytest.mark.parametrize("low", [-22.0, -26.0, -29.0])
def test_many_small_weights_add_up(H, low):
    """One key takes nearly all the weight and has the value 0; 4200 keys at 2^low have 1.

    A weight is off by at most 2^-11 of itself or 2^-32 of the largest, a score's exponent by
    2^-22 of it (the scale's two roundings and the product's), the output's rounding 2^-8."""
    r = np.random.default_rng(40)
    n = 4201
    x = low - 0.25 * r.integers(0, 4, n)
    x[n // 3] = 0.0
    v = np.ones(n)
    v[n // 3] = 0.0
    s = exact_scores(H, x, v, n - 1)
    p = np.exp(x * s["scale"])
    ref = (p * v).sum() / p.sum()
    tol = ((np.maximum(2.0 ** -11 * p, 2.0 ** -32) + 2.0 ** -21 * np.abs(x) * p) * v).sum() / p.sum()
    out = base.run(s)[0]
    assert (np.abs(out[:, 0] - ref) <= tol * 1.01 + 2.0 ** -8 * ref).all(), (out[0, 0], ref, tol)
    assert (out[:, 1:] == 0).all()


def staircase(H, n=200, prefix=1400, block=128):
    """Scores that climb by 10, 5 or 20 (in log2) from a block of keys to the next, or fall by
    10, by groups of eight rows: the accumulator is rescaled at every block, at every second
    one, or never, for rows that share a warp.  Value column k is zero outside block k of the
    keys, so every block's share of the output is compared by itself.

    Scores and values are exact; a weight is off by 2^-11 of itself or 2^-32 of the row's
    largest, exponents by 2^-22 of the largest score (in a weight and in the sum), the output's
    rounding is 2^-8.  Returns the batch, its scores (log2), values, output and tolerance."""
    r = np.random.default_rng(41)
    keys = n + prefix
    j = np.arange(keys)
    x = 10.0 * (j // block) + r.integers(0, 4, keys)
    s = exact_scores(H, x, np.zeros(keys), prefix, n - 1)
    at = s["rows"][0]
    v = torch.from_numpy(r.uniform(0.5, 2.0, keys)).bfloat16()
    s["c_kv"][at, 8 + torch.from_numpy(j // block)] = v
    a = np.array([1.0, 0.5, 2.0, -1.0])[np.arange(n) // 8 % 4]
    s["q_nope"][:, :, 0] = torch.from_numpy(a).bfloat16()[:, None]
    y = a[:, None] * x[None] * s["scale"] / np.log(2.0)
    y[j[None] > prefix + np.arange(n)[:, None]] = -np.inf
    p = np.exp2(y - y.max(1, keepdims=True))
    V = np.zeros((keys, 56))
    V[j, j // block] = v.double().numpy()
    l = p.sum(1, keepdims=True)
    ref = p @ V / l
    rel = 2.0 ** -11 + 2.0 ** -20 * np.abs(a[:, None] * x.max())
    tol = (rel * (p @ V) + (p > 0).astype(float) @ V * 2.0 ** -32) / l * 1.01 + 2.0 ** -8 * ref
    return s, y, V, ref, tol


@pytest.mark.parametrize("H", [1, 160])     # cut along the keys, whole items
def test_moving_maxima_block_by_block(H):
    s, _, _, ref, tol = staircase(H)
    out = base.run(s)
    for h in (0, H - 1):
        assert (np.abs(out[:, h, :56] - ref) <= tol).all(), (h, np.abs(out[:, h, :56] - ref).max())
        assert (out[:, h, 56:] == 0).all()
