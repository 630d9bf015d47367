"""GPU tests of tv_shared_attn against plain attention over every sequence's keys in 64 bits.

Tolerance.  The softmax weights are rounded to bf16 and so may be the output: h = 2^-8 relative
each.  Everything else is 32-bit: a score is a sum of 36 accumulations of products of 16 (counted
as 64 roundings of 2^-23, accumulations being cut, of S = the largest scale sum |q||k|), and an
output one of n/16 accumulations (and 80 more for rescaling, joining and the division).  With
A = sum_j p_j |c_j| an element is within
    A (h + 3 * 64 * 2^-23 S + (n/16 + 80) 2^-23) + h |out|
and a row's lse within 64 * 2^-23 S + (n/64 + 64) 2^-23.  For independent normal keys the
roundings of weights and output are independent, of rms below h/sqrt(3) each: a row's error is
of rms below 0.82 h of the row's rms, and h is asked of it.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import decode_model as dm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
H_STEP, F_STEP = 2.0 ** -8, 2.0 ** -23


def make(seed, members, shared, own, H=16, Q=1, paged=True, tree=True, q_scale=0.25, ungrouped=0,
         spare=2):
    """Sequences in groups; `ungrouped` more share nothing but are a group each.  Cache rows that
    hold no key are NaN."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    members = list(members) + [1] * ungrouped
    shared = list(shared) + [0] * ungrouped
    B = sum(members)
    group = np.repeat(np.arange(len(members)), members)
    start = np.concatenate([[0], np.cumsum(members)])
    extra = r.integers(0, own + 1, B) if np.isscalar(own) else np.asarray(own)
    prefix = np.array([shared[group[b]] + extra[b] for b in range(B)], np.int64)
    need = -(-(prefix + Q) // 64)
    whole = [s // 64 for s in shared]

    def randn(*shape, s=1.0):
        return (torch.randn(shape, generator=g) * s).bfloat16()

    if paged:
        num = sum(whole) + int(sum(need[b] - whole[group[b]] for b in range(B))) + spare
        perm = r.permutation(num)
        table = np.full((B, int(need.max()) + 1), -1, np.int32)
        at = 0
        for i, w in enumerate(whole):
            table[start[i]:start[i + 1], :w] = perm[at:at + w]
            at += w
        for b in range(B):
            n = int(need[b]) - whole[group[b]]
            table[b, whole[group[b]]:need[b]] = perm[at:at + n]
            at += n
        stride, rows = 0, num * 64
    else:
        table, stride = None, int((prefix + Q).max()) + 5
        rows = B * stride
    c = torch.full((rows, 512), float("nan"), dtype=torch.bfloat16)
    k = torch.full((rows, 64), float("nan"), dtype=torch.bfloat16)
    common = [(randn(s, 512), randn(s, 64)) for s in shared]
    keys = []
    for b in range(B):
        n = int(prefix[b]) + Q
        j = np.arange(n)
        at = table[b, j // 64].astype(np.int64) * 64 + j % 64 if paged else b * stride + j
        cs, ks = common[group[b]]
        mine = n - len(cs)
        keys.append((torch.cat([cs, randn(mine, 512)]), torch.cat([ks, randn(mine, 64)])))
        c[at], k[at] = keys[b]
    vis = np.zeros((B, Q, Q), bool)
    for b in range(B):
        for i in range(Q):
            if not tree:
                vis[b, i, :i] = True
            elif i:
                vis[b, i] = vis[b, r.integers(0, i)]
            vis[b, i, i] = True
    bits = (vis.astype(np.uint64) << np.arange(Q, dtype=np.uint64)).sum(-1).astype(np.uint64)
    return dict(H=H, Q=Q, B=B, q_latent=randn(B, Q, H, 512, s=q_scale), q_pe=randn(B, Q, H, 64),
                c_kv=c, k_pe=k, table=table, stride=stride, prefix=prefix, start=start,
                shared=shared, keys=keys, vis=vis, anc=bits.view(np.int64) if tree else None,
                scale=192 ** -0.5)


def device(s, out=torch.bfloat16):
    def put(a, dt=np.int32):
        return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dt)).cuda()
    rows = (s["B"], s["Q"], s["H"])
    return dict(q_latent=s["q_latent"].cuda(), q_pe=s["q_pe"].cuda(), c_kv=s["c_kv"].cuda(),
                k_pe=s["k_pe"].cuda(), table=put(s["table"]), prefix=put(s["prefix"]),
                start=put(s["start"]), shared=put(s["shared"]), anc=put(s["anc"], np.int64),
                out=torch.full((*rows, 512), -77.0, dtype=out, device="cuda"),
                lse=torch.full(rows, -77.0, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def launch(s, d, **kw):
    p = dict(max_prefix_len=int(max(0, s["prefix"].max())), anc=d["anc"], page_table=d["table"],
             kv_stride_b=s["stride"], status=d["status"], group_start=d["start"],
             shared_len=d["shared"], lse=d["lse"])
    p.update(kw)
    tv.shared_attn(d["q_latent"], d["q_pe"], d["c_kv"], d["k_pe"], d["prefix"],
                   p.pop("group_start"), p.pop("shared_len"), d["out"], p.pop("lse"), s["scale"],
                   **p)


def poisoned_workspace(s, d):
    a = tv.shared_args(d["q_latent"], d["q_pe"], d["c_kv"], d["k_pe"], d["prefix"], d["start"],
                       d["shared"], d["out"], d["lse"], s["scale"], int(s["prefix"].max()),
                       d["anc"], d["table"], 64, s["stride"])
    return torch.full((tv.shared_workspace_size(a),), 255, dtype=torch.uint8, device="cuda")


def run(s, out=torch.bfloat16, status=0, **kw):
    d = device(s, out)
    launch(s, d, workspace=poisoned_workspace(s, d), **kw)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == status
    return d


def visible(s, b, n):
    v = torch.ones((s["Q"], n), dtype=torch.bool, device="cuda")
    v[:, n - s["Q"]:] = torch.from_numpy(s["vis"][b]).cuda()
    return v


def close(s, d, sequences=None, rms=True):
    for b in range(s["B"]) if sequences is None else sequences:
        c, k = (t.cuda() for t in s["keys"][b])
        n = len(c)
        ref, lse, A, S = dm.attention(d["q_latent"][b], d["q_pe"][b], c, k, visible(s, b, n),
                                      s["scale"])
        got, got_lse = d["out"][b].double(), d["lse"][b].double()
        assert torch.isfinite(got).all() and torch.isfinite(got_lse).all()
        h_out = H_STEP if d["out"].dtype is torch.bfloat16 else F_STEP
        rel = H_STEP + 3 * 64 * F_STEP * S[..., None] + (n / 16 + 80) * F_STEP
        over = (got - ref).abs() - (A * rel + h_out * ref.abs())
        assert over.max() <= 0, (b, float(over.max()))
        off = (got_lse - lse).abs() - (64 * F_STEP * S + (n / 64 + 64) * F_STEP)
        assert off.max() <= 0, (b, float(off.max()))
        if rms and n >= 64:
            err = ((got - ref) ** 2).mean(-1).sqrt() / (ref ** 2).mean(-1).sqrt()
            assert err.max() <= H_STEP, (b, float(err.max()))


CASES = [
    # one token over an empty prefix; a short prompt; a page that ends at the last key
    dict(members=[1], shared=[0], own=[0], H=1),
    dict(members=[1], shared=[0], own=[63], H=1),
    dict(members=[4], shared=[700], own=40),
    dict(members=[8], shared=[2048], own=[0, 1, 62, 63, 64, 65, 127, 128]),
    # odd heads, trees, a prefix that ends inside a page, one below a page, one user alone
    dict(members=[3, 1, 5], shared=[641, 129, 63], own=200, H=5, Q=3),
    dict(members=[5, 2], shared=[1000, 320], own=100, H=33, Q=9),
    # rows that fill tiles by themselves: nothing to gain
    dict(members=[2, 2], shared=[0, 1024], own=90, H=64, Q=2),
    dict(members=[3], shared=[400], own=30, H=128, Q=1),
    # queries as a chain; the most of them
    dict(members=[2, 3], shared=[256, 515], own=70, H=2, Q=17, tree=False),
    dict(members=[3], shared=[1300], own=20, H=3, Q=64),
    # a contiguous cache
    dict(members=[6], shared=[1100], own=50, paged=False),
    dict(members=[2, 3], shared=[64, 700], own=130, H=7, Q=5, paged=False),
    # many sequences alone, and many in one group
    dict(members=[40], shared=[500], own=10, H=1, ungrouped=25),
    # long keys: several pieces a tile
    dict(members=[9], shared=[9000], own=3000, H=16),
    dict(members=[1], shared=[0], own=[15000], H=4),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_plain_attention(i):
    s = make(100 + i, **CASES[i])
    close(s, run(s), sequences=range(0, s["B"], max(1, s["B"] // 12)))


@pytest.mark.parametrize("i", [2, 4, 13])
def test_float32_output(i):
    s = make(200 + i, **CASES[i])
    close(s, run(s, torch.float32))


def test_one_key_is_its_value():
    s = make(1, [3], [0], [0, 0, 0], H=5)
    d = run(s)
    for b in range(3):
        assert torch.equal(d["out"][b, 0].cpu(), s["keys"][b][0].expand(5, 512))


def test_sharp_and_moving_maxima():
    # scores that grow along the keys, so that every block moves the maximum, and sharp ones
    s = make(2, [6], [1500], 60, q_scale=2.0)
    for b in range(s["B"]):
        c = s["keys"][b][0]
        at = torch.from_numpy(s["table"][b, np.arange(len(c)) // 64].astype(np.int64) * 64 +
                              np.arange(len(c)) % 64)
        c[:, 0] = (torch.arange(len(c)) * (8.0 / 1500)).bfloat16()
        s["c_kv"][at] = c
    s["q_latent"][..., 0] = 40.0
    close(s, run(s), rms=False)


def test_no_groups_and_no_lse():
    s = make(3, [4], [512], 60)
    a, b = run(s), run(s, group_start=None, shared_len=None)
    close(s, b)
    c = device(s)
    launch(s, c, lse=None)
    torch.cuda.synchronize()
    assert torch.equal(c["out"], a["out"])


def test_shared_keys_come_from_the_first_sequence():
    s = make(4, [12], [1280], 30)
    s["table"][1:, :1280 // 64] = -1
    close(s, run(s))


def test_rows_that_see_nothing():
    s = make(5, [2, 2], [0, 640], [0, 5, 9, 0], H=3, Q=4)
    s["anc"][0] = 0          # an invalid tree over no prefix
    s["anc"][2] = 0          # and over one: the prefix alone is left
    s["vis"][0] = s["vis"][2] = False
    d = run(s)
    assert (d["out"][0] == 0).all() and (d["lse"][0] == -math.inf).all()
    close(s, d, [1, 2, 3])


def test_out_of_bounds_sequences():
    s = make(6, [3, 4], [300, 1280], 40)
    good = run(s)
    bad = dict(s, prefix=s["prefix"].copy())
    bad["prefix"][1], bad["prefix"][5] = -3, 10 ** 6
    d = device(bad)
    launch(bad, d, max_prefix_len=int(s["prefix"].max()),
           workspace=poisoned_workspace(s, device(s)))
    torch.cuda.synchronize()
    assert int(d["status"].item()) == tv.TV_ERR_BOUNDS
    for b in (1, 5):
        assert (d["out"][b] == 0).all() and (d["lse"][b] == -math.inf).all()
    close(s, d, [0, 2, 3, 4, 6])
    assert torch.equal(d["out"][6], good["out"][6])


@pytest.mark.parametrize("start,shared", [
    ([0, 3, 6], [300, 1280]), ([1, 3, 7], [300, 1280]), ([0, 8, 7], [300, 1280]),
    ([0, -1, 7], [300, 1280]), ([0, 3, 7], [300, 1321]), ([0, 3, 7], [-1, 1280]),
    ([0, 3, 7], [300, 2 ** 31 - 1])])
def test_groups_that_are_not(start, shared):
    s = make(7, [3, 4], [300, 1280], 40)
    d = device(dict(s, start=np.array(start), shared=np.array(shared)))
    launch(s, d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == tv.TV_ERR_BOUNDS
    close(s, d)


def test_empty_groups():
    s = make(8, [3, 4], [300, 1280], 40)
    d = device(dict(s, start=np.array([0, 0, 3, 3, 7, 7]), shared=np.array([5, 300, 9, 1280, 0])))
    launch(s, d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    close(s, d)


def test_pages_outside_the_cache_read_as_zeros():
    s = make(9, [8], [1280], [100] * 8)
    s["table"][0, 3], s["table"][4, 20] = 10 ** 6, -7
    for b in range(8):
        s["keys"][b][0][192:256] = 0
        s["keys"][b][1][192:256] = 0
    for t in s["keys"][4]:
        t[1280:1344] = 0
    close(s, run(s, status=tv.TV_ERR_BOUNDS))


def test_same_bits_again_and_in_graphs():
    s = make(10, [20, 1, 7], [3000, 100, 700], 600)
    a = run(s)
    d = device(s)
    launch(s, d)
    torch.cuda.synchronize()
    one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    e = device(s)
    with torch.cuda.graph(one):
        launch(s, d)
    with torch.cuda.graph(two):
        launch(s, e)
    for t in (d, e):
        t["out"].fill_(0)
    # two graphs side by side: each has its own workspace
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        one.replay()
        with torch.cuda.stream(side):
            two.replay()
    torch.cuda.synchronize()
    for t in (d, e):
        assert torch.equal(t["out"], a["out"]) and torch.equal(t["lse"], a["lse"])


def test_graph_follows_its_lengths():
    s = make(11, [12], [1280], 200)
    d = device(s)
    launch(s, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch(s, d)
    d["prefix"] -= 30      # fewer own keys, the last 30 of the prefix now unseen
    d["prefix"].clamp_(min=1280)
    d["prefix"].copy_(torch.minimum(d["prefix"], torch.from_numpy(s["prefix"]).cuda().int()))
    graph.replay()
    torch.cuda.synchronize()
    new = d["prefix"].cpu().numpy()
    t = dict(s, prefix=new, keys=[(c[:n + 1], k[:n + 1]) for (c, k), n in zip(s["keys"], new)])
    close(t, d)


def test_cache_rows_within_wider_ones():
    s = make(15, [6, 2], [1280, 70], 60, Q=2, H=8)
    want, d = run(s), device(s)
    wide = torch.full((len(s["c_kv"]), 608), float("nan"), dtype=torch.bfloat16, device="cuda")
    d["c_kv"], d["k_pe"] = wide[:, 8:520], wide[:, 536:600]
    d["c_kv"].copy_(s["c_kv"])
    d["k_pe"].copy_(s["k_pe"])
    launch(s, d)
    torch.cuda.synchronize()
    assert torch.equal(d["out"], want["out"]) and torch.equal(d["lse"], want["lse"])


def test_keys_that_are_not_finite_stay_in_their_sequence():
    # (own keys of one sequence; the shared ones belong to all)
    s = make(16, [8], [1280], [90] * 8)
    d = device(s)
    page = int(s["table"][3, 21])
    d["c_kv"][page * 64 + 5] = float("nan")
    launch(s, d)
    torch.cuda.synchronize()
    # (a key's latent row is part of its score, q . c + q_pe . k, so the sum is NaN as well)
    assert torch.isnan(d["out"][3]).all() and torch.isnan(d["lse"][3]).all()
    close(s, d, [0, 1, 2, 4, 5, 6, 7])
    d["k_pe"][page * 64 + 5] = float("inf")
    launch(s, d)
    torch.cuda.synchronize()
    close(s, d, [0, 1, 2, 4, 5, 6, 7])


def test_on_another_stream():
    s = make(12, [5], [640], 60)
    a, d = run(s), device(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    launch(s, d, stream=side)
    side.synchronize()
    assert torch.equal(d["out"], a["out"])


def test_more_sequences_than_threads():
    s = make(13, [700, 600], [128, 320], 3, H=1)
    close(s, run(s), range(0, 1300, 83))


def test_waits_end_and_the_next_call_is_whole():
    s = make(14, [6], [1280], 60)
    want = run(s)
    d = device(s)
    counts = torch.zeros(2, dtype=torch.int32, device="cuda")
    lib = tv.load()
    try:
        assert lib.tv_testing_set_shared_fault(1, 10_000_000,
                                               ctypes.c_void_p(counts.data_ptr())) == tv.TV_OK
        launch(s, d)
        torch.cuda.synchronize()
    finally:
        lib.tv_testing_set_shared_fault(0, 0, None)
    assert int(d["status"].item()) == tv.TV_ERR_TIMEOUT
    left, aborted = counts.tolist()
    assert left > 0 and aborted > 0 and left % 2 == 0
    close(s, run(s))
    assert torch.equal(run(s)["out"], want["out"])
