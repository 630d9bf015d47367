"""GPU tests of tv_token_sample against its rule in 64 bits.

Tokens and counts have to be equal.  The library's weights are off by 2^-36 of themselves and
5/8 of a unit of 2^-44, so a draw or a cut may differ where a uniform number or a share falls that
near to a boundary: with at most 2^18 boundaries in a row, that is one row in 10^5 or fewer of
random inputs.  Inputs here are seeded, a few thousand rows in all.
"""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import decode_model as dm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]


def sample(logits, u, status=0, **kw):
    """(tokens, kept) of logits (a CUDA tensor); filters as numbers or lists."""
    B = logits.shape[0]

    def row(v, dt):
        if v is None:
            return None
        a = np.broadcast_to(np.asarray(v, np.float64), (B,)).copy()
        return torch.from_numpy(a).to(dt).cuda()
    tokens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    kept = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.token_sample(logits, row(u, torch.float32), tokens,
                    temperature=row(kw.get("temperature"), torch.float32),
                    top_k=row(kw.get("k"), torch.int32), top_p=row(kw.get("p"), torch.float32),
                    min_p=row(kw.get("m"), torch.float32), kept=kept, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return tokens.cpu().numpy(), kept.cpu().numpy()


def check(logits, u, **kw):
    B = logits.shape[0]
    x = logits.double().cpu().numpy()
    got = sample(logits.cuda(), u, **kw)
    names = dict(temperature=1.0, k=0, p=1.0, m=0.0)
    args = {n: np.broadcast_to(kw.get(n, d), (B,)) for n, d in names.items()}
    us = np.broadcast_to(u, (B,))
    for b in range(B):
        want = dm.next_token(x[b], us[b], *(args[n][b] for n in names))
        assert (got[0][b], got[1][b]) == want, (b, {n: args[n][b] for n in names})


def rows(seed, B, V, dt=torch.float32, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((B, V), generator=g) * spread).to(dt), \
        torch.rand(B, generator=g).numpy()


FILTERS = [dict(), dict(k=1), dict(k=40), dict(p=0.9), dict(m=0.1), dict(k=300, p=0.7),
           dict(k=50, p=0.95, m=0.02), dict(p=0.5, m=0.001), dict(k=10 ** 9, p=0.999),
           dict(temperature=0.3, p=0.98), dict(temperature=2.0, k=1000, m=0.2),
           dict(temperature=0.0, k=5)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("f", range(len(FILTERS)))
@pytest.mark.parametrize("B,V", [(7, 1), (5, 3), (9, 129), (6, 5003), (3, 32000)])
def test_against_the_rule(B, V, f, dt):
    x, u = rows(B * 1000 + f, B, V, dt)
    check(x, u, **FILTERS[f])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,V,spread", [(2, 163840, 3.0), (40, 50257, 1.0), (1, 1 << 18, 1.5),
                                        (300, 4096, 4.0)])
def test_mixed_rows(B, V, spread, dt):
    x, u = rows(V, B, V, dt, spread)
    i = np.arange(B)
    check(x, u, temperature=np.where(i % 5 == 4, 0.0, 0.8 + 0.05 * (i % 7)),
          k=np.where(i % 3 == 0, 1 + 17 * i, 0), p=np.where(i % 2 == 0, 0.93, 1.0),
          m=np.where(i % 4 == 1, 0.01, 0.0))


@pytest.mark.parametrize("B", [200, 512, 513, 1300])
def test_more_rows_than_fit_at_once(B):
    # long and short rows in any order, rows that are refused among them
    logits, u = rows(17, B, 300)
    g = np.random.default_rng(17)
    pick = lambda *v: g.choice(v, B)
    kw = dict(temperature=pick(1.0, 0.7, 0.0), k=pick(0, 0, 7, 400), p=pick(1.0, 0.9, 0.5),
              m=pick(0.0, 0.0, 0.01))
    check(logits, u, **kw)
    kw["temperature"][::3] = -1.0
    tokens, kept = sample(logits.cuda(), u, status=tv.TV_ERR_INVALID_ARG, **kw)
    assert (tokens[::3] == -1).all() and (kept[::3] == 0).all()
    assert (np.delete(kept, np.s_[::3]) > 0).all()


@pytest.mark.parametrize("V", [64, 4096, 131072])
def test_equal_logits(V):
    # n equal weights: sums are exact, a draw is floor(u n), a nucleus ceil(p n), by index
    x = torch.full((6, V), -2.5)
    u = np.array([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24, 0.5 - 2.0 ** -24])
    t, n = sample(x.cuda(), u)
    assert t.tolist() == [int(v * V) for v in u] and n.tolist() == [V] * 6
    t, n = sample(x.cuda(), u, p=0.25)
    assert n.tolist() == [V // 4] * 6 and t.tolist() == [int(v * (V // 4)) for v in u]
    t, n = sample(x.cuda(), u, k=V // 2, p=0.25)
    assert n.tolist() == [V // 8] * 6 and t.tolist() == [int(v * (V // 8)) for v in u]
    t, n = sample(x.cuda(), u, k=24, m=1.0)
    assert n.tolist() == [24] * 6 and t.tolist() == [int(np.float32(v) * 24.0) for v in u]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B", [6, 160])
def test_as_many_equal_logits_as_there_can_be(B, dt):
    # the sums of 2^18 of the largest weights need all but two bits; 160 rows: one CTA each
    V = 1 << 18
    g = torch.Generator().manual_seed(21)
    x = torch.full((6, V), 0.5)
    x[1, ::7] = 0.25
    x[2] = 0.25 * torch.randint(0, 2, (V,), generator=g)
    x[3, :3000] = torch.randn(3000, generator=g) - 1
    x[4, 1::3] = -0.0
    x[5] = torch.where(torch.rand(V, generator=g) < 0.7, 0.5, -3.0)
    u = np.array([0.9, 0.3, 0.99999, 0.5, 0.7, 0.1])
    for kw in (dict(p=[0.9, 0.95, 0.75, 0.99, 0.9999, 0.9999]), dict(k=[200000] * 6),
               dict(k=[150000, 224695, 140000, 262143, 200000, 190000], p=[0.6] * 6)):
        want = [dm.next_token(x[b].double().numpy(), u[b], 1.0, kw.get("k", [0] * 6)[b],
                              kw.get("p", [1.0] * 6)[b], 0.0) for b in range(6)]
        rep = np.arange(B) % 6
        kw = {n: np.array(v)[rep] for n, v in kw.items()}
        got = sample(x.to(dt).cuda()[torch.from_numpy(rep).cuda()], u[rep], **kw)
        assert [(t, n) for t, n in zip(*got)] == [want[b] for b in rep]


def test_ties_at_the_cut_go_to_the_lowest_index():
    # few distinct values, many times each
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-4, 4, (24, 20001), generator=g).float()
    u = torch.rand(24, generator=g).numpy()
    i = np.arange(24)
    check(x, u, k=np.where(i % 3 == 0, 7 + 313 * i, 0),
          p=np.where(i % 3 == 1, 0.02 + 0.04 * i, 1.0), m=np.where(i % 3 == 2, 0.3, 0.0))
    check(x.bfloat16(), u, k=3000 + 100 * i, p=0.3 + 0.02 * i)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_shares_next_to_the_edge_of_ties(dt):
    # two values, many times each: estimates of the sums from few bins are off by up to 0.4 %,
    # and the share falls that near to where the first value's tokens end
    g = torch.Generator().manual_seed(15)
    for gap in (0.5, 0.503, 0.5078125, 1.25, 3.0):
        x = torch.full((16, 9000), 2.0)
        x[:, torch.randperm(9000, generator=g)[:5000]] = 2.0 - gap
        x = x.to(dt)
        w = np.exp(x.double().numpy()[0])
        first = w[w == w.max()].sum() / w.sum()
        p = first * (1 + np.linspace(-0.004, 0.004, 16))
        check(x, torch.rand(16, generator=g).numpy(), p=p)


def test_around_zero_and_far_apart():
    # the cut falls between values whose bit patterns lie far apart, signed zeros among them
    g = torch.Generator().manual_seed(6)
    x = torch.randn((8, 3001), generator=g) * 1e-6
    x[:, ::7] = 0.0
    x[:, 3::11] = -0.0
    x[4:] *= 1e30
    u = torch.rand(8, generator=g).numpy()
    for kw in (dict(k=1500), dict(p=0.5), dict(k=2000, p=0.4),
               dict(temperature=1e-6, k=1000), dict(temperature=1e20, p=0.7)):
        check(x, u, **kw)
    y = torch.tensor([[3e38, -3e38, 1e38, 2.0, -2.0]]).repeat(3, 1)
    check(y, [0.0, 0.5, 0.99], k=4)
    check(y, [0.0, 0.5, 0.99], temperature=1e30, k=4, p=0.8)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1.0, 7.0])
def test_logits_on_a_grid(dt, T):
    # all of a bin's tokens on the same side of its middle, those of the upper bins on the other
    # one: the running sums' estimate is off by more than chance would have it
    g = torch.Generator().manual_seed(19)
    width = 48 / 4095 * math.log(2) * T
    j = torch.randint(0, 400, (1, 40000), generator=g).double()
    x = -(j + torch.where(j < 100, 0.03, 0.97)) * width
    x[0, 7] = 0.0
    p = np.concatenate([np.linspace(0.02, 0.98, 40), [0.999, 0.9999]])
    u = torch.rand(len(p), generator=g).numpy()
    check(x.to(dt).repeat(len(p), 1), u, p=p, temperature=T)


@pytest.mark.parametrize("V", [50257, 200000])
def test_cuts_among_many_equal_bf16_logits(V):
    # a few values, each some hundred to some ten thousand times
    logits, u = rows(20, 10, V, torch.float32, 1.0)
    x = logits * torch.tensor([0.5, 1, 3, 0.1, 0.02, 1, 1, 3, 0.5, 1])[:, None]
    x[5:] = (x[5:] * 4).round() / 4 - 2
    p = np.array([0.9, 0.95, 0.3, 0.5, 0.7, 0.2, 0.99, 0.9, 0.6, 0.01])
    check(x.to(torch.bfloat16), u, p=p)
    check(x.to(torch.bfloat16), u, p=p, m=0.01, k=[0, 5000, 0, V // 2, 0, 0, 30000, 0, 900, 0])


@pytest.mark.parametrize("f", [dict(), dict(p=0.9), dict(k=900, p=0.8), dict(p=0.99, m=1e-4)])
def test_bf16_values_of_any_size(f):
    # the weights of a row's values are taken from a table, those of values next to 0 are not:
    # negative maxima, tiny ones, rows far from 0, rows around it, wide and narrow ones
    B, V = 12, 30011
    logits, u = rows(18, B, V, torch.float32, 1.0)
    spread = torch.tensor([3, 3, 3, 1e-3, 1e-6, 2, 2, 300, 0.1, 5, 3, 3.0])[:, None]
    shift = torch.tensor([-20, 0, 40, 0, 0, 1000, -1000, 0, -0.6, 0, 0, -13.2])[:, None]
    t = np.array([1, 1, 1, 1, 1e-7, 1, 1, 40, 0.05, 0.1, 30, 1.0])
    x = logits * spread + shift
    x[9] = x[9] * (torch.arange(V) % 3 == 0)          # zeros
    x[10, ::2] = torch.randn(len(x[10, ::2]), generator=torch.Generator().manual_seed(1)) * 1e-30
    x[11] = -x[11].abs() * 1e-3                        # none above 0, the largest next to it
    x[1, ::5] = float("-inf")
    check(x.to(torch.bfloat16), u, temperature=t, **f)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_draws_next_to_boundaries(dt):
    # uniforms at the two floats around a boundary of the running sums, where they are farther
    # from it than the weights' errors could move it (2^-36)
    g = torch.Generator().manual_seed(16)
    for V, kw in ((3000, {}), (3000, dict(k=700)), (40000, dict(p=0.8))):
        x = (torch.randn((1, V), generator=g) * 2).to(dt)
        x64 = x[0].double().numpy()
        w = np.exp(x64 - x64.max())
        n = dm.next_token(x64, 0.5, 1.0, kw.get("k", 0), kw.get("p", 1.0))[1]
        chosen = np.sort(np.argsort(-x64, kind="stable")[:n])
        edges = (np.cumsum(w[chosen]) / w[chosen].sum())[:-1]
        edges = edges[:: max(1, len(edges) // 200)]
        below = edges.astype(np.float32)
        below = np.where(below > edges, np.nextafter(below, np.float32(0)), below)
        u = np.concatenate([below, np.nextafter(below, np.float32(1))])
        far = np.abs(u.astype(np.float64) - np.concatenate([edges, edges])) > 2.0 ** -36
        u = u[far & (u < 1)]
        check(x.repeat(len(u), 1), u, **kw)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_masked_tokens(dt):
    x, u = rows(7, 6, 4099, dt)
    x[:, ::2] = -float("inf")
    x[5, 1:] = -float("inf")
    x[5, 0] = 1.0
    for kw in (dict(), dict(k=4000), dict(k=100), dict(p=0.9), dict(k=3000, p=0.9, m=0.001)):
        check(x, u, **kw)


def test_weights_below_a_unit_are_kept_in_order():
    # 50 log2 units below the largest a weight is nothing, but top-k still counts the token
    x = torch.tensor([[0.0, -60.0, -50.0, -40.0, -70.0, -60.0, -55.0]] * 2)
    t, n = sample(x.cuda(), [0.0, 0.99], k=[5, 6])
    assert t.tolist() == [0, 0] and n.tolist() == [5, 6]


@pytest.mark.parametrize("off", [1, 3, 5])
def test_rows_at_any_alignment(off):
    x, u = rows(8, 5, 7001 + off, torch.bfloat16)
    check(x[:, off:], u, p=0.9)
    y = torch.empty((5, 9001)).normal_(generator=torch.Generator().manual_seed(off)).cuda()
    part = y[:, off:off + 8003]
    a = sample(part, u, k=99, p=0.8)
    b = sample(part.contiguous(), u, k=99, p=0.8)
    assert a[0].tolist() == b[0].tolist() and a[1].tolist() == b[1].tolist()


def test_edges_of_the_filters():
    x, u = rows(9, 8, 1000)
    want = torch.argmax(x, 1).tolist()
    for kw in (dict(k=1), dict(p=0.0), dict(p=-1.0), dict(p=1e-30), dict(m=1.0), dict(m=7.0),
               dict(k=1, p=0.1, m=0.9)):
        t, n = sample(x.cuda(), u, **kw)
        assert t.tolist() == want and n.tolist() == [1] * 8, kw
    for kw in (dict(k=0), dict(k=-5), dict(k=1000), dict(p=1.0), dict(p=3.0), dict(m=0.0),
               dict(m=-1.0)):
        t, n = sample(x.cuda(), u, **kw)
        assert n.tolist() == [1000] * 8, kw
    # uniform numbers outside [0, 1): the nearest inside
    a = sample(x.cuda(), [-1.0, float("nan"), 1.0, 2.0, float("inf"), -float("inf"), 0.0,
                          1 - 2.0 ** -24])[0]
    b = sample(x.cuda(), [0.0, 0.0, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 1 - 2.0 ** -24, 0.0, 0.0,
                          1 - 2.0 ** -24])[0]
    assert a.tolist() == b.tolist()


@pytest.mark.parametrize("V", [5, 40000])
def test_bad_rows(V):
    x, u = rows(10, 8, V)
    x[1, V // 2] = float("nan")
    x[2] = -float("inf")
    x[3, 0] = float("inf")
    temp = [1.0, 1.0, 1.0, 1.0, -1.0, float("nan"), 1.0, 0.0]
    p = [0.9, 0.9, 0.9, 0.9, 0.9, 0.9, float("nan"), float("nan")]
    t, n = sample(x.cuda(), u, status=tv.TV_ERR_INVALID_ARG, temperature=temp, p=p)
    assert t[1:7].tolist() == [-1] * 6 and n[1:7].tolist() == [0] * 6
    assert (t[0], n[0]) == dm.next_token(x[0].numpy(), u[0], 1.0, 0, 0.9)
    assert (t[7], n[7]) == (int(torch.argmax(x[7])), 1)      # greedy rows read no filters


def test_a_row_is_the_same_in_any_batch():
    # the number of CTAs of a row changes with the batch
    x, u = rows(11, 700, 20000, torch.bfloat16, 2.0)
    x = x.cuda()
    for kw in (dict(p=0.9), dict(k=500, p=0.8), dict()):
        t, n = sample(x, u, **kw)
        for b in (0, 13, 699):
            a = sample(x[b:b + 1], u[b:b + 1], **kw)
            assert (a[0][0], a[1][0]) == (t[b], n[b])


def test_in_a_graph_with_new_inputs():
    x, u = rows(12, 16, 30000)
    xs, us = x.cuda(), torch.from_numpy(u).cuda()
    tokens = torch.zeros(16, dtype=torch.int32, device="cuda")
    p = torch.full((16,), 0.9, device="cuda")
    k = torch.full((16,), 60, dtype=torch.int32, device="cuda")
    tv.token_sample(xs, us, tokens, top_p=p, top_k=k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.token_sample(xs, us, tokens, top_p=p, top_k=k)
    y, v = rows(13, 16, 30000)
    xs.copy_(y)
    us.copy_(torch.from_numpy(v))
    p.fill_(0.6)
    k.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want = [dm.next_token(y[b].numpy(), v[b], 1.0, 0, 0.6)[0] for b in range(16)]
    assert tokens.tolist() == want


def test_distribution():
    # 2^16 draws of one row, evenly spaced uniforms: every kept token as often as its share
    x = torch.randn((1, 50), generator=torch.Generator().manual_seed(14)) * 1.5
    n = 1 << 16
    u = (np.arange(n) + 0.5) / n
    t, kept = sample(x.repeat(n, 1).cuda(), u.astype(np.float32), p=0.9)
    w = np.exp(x[0].double().numpy())
    order = np.argsort(-w)[:kept[0]]
    share = np.zeros(50)
    share[order] = w[order] / w[order].sum()
    # (evenly spaced: a count is off by less than one at each end, and float32 uniforms by
    # half a step)
    assert np.abs(np.bincount(t, minlength=50) - n * share).max() <= 2.0
