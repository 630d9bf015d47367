"""GPU tests of tv_tree_sample against its plain statement in 64 bits.

The outputs are integers and have to be equal.  The kernel's sums are exact in units of
2^-44 of a row's largest weight, its weights good to 2^-38, so a uniform number would have
to fall within about 2^-37 of one of the boundaries it is compared with; with the fewer than
2^24 boundaries of all these cases that happens in one of 2^13 sets of seeds, and the seeds
are fixed.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import serving_model as sm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]


def make(seed, B, Q, V, dtype="fp32", draft=None, spread=3.0, sharp=2.0, wide=6):
    """Inputs of a call: trees whose children are the drafter's best tokens or a draw of it
    without replacement, and target logits near the drafter's."""
    r = np.random.default_rng(seed)
    parent = np.full((B, Q), -1, np.int32)
    tokens = np.zeros((B, Q), np.int32)
    by_node = draft == "node"
    logq = r.normal(size=(B, Q, V)) * spread          # one row per node, or per depth
    logq -= np.log(np.exp(logq).sum(-1, keepdims=True))
    depth = np.zeros((B, Q), np.int64)
    rows = np.zeros((B, Q), np.int64)
    for b in range(B):
        order = {}
        for i in range(1, Q):
            p = int(r.integers(max(0, i - wide), i))
            while len(order.get(p, [1])) == 0:
                p += 1
            parent[b, i], depth[b, i] = p, depth[b, p] + 1
            row = p if by_node else depth[b, p]
            if p not in order:
                score = logq[b, row] + (r.gumbel(size=V) if draft else 0)
                order[p] = np.argsort(-score).tolist()
            tokens[b, i] = order[p].pop(0)
        rows[b] = np.arange(Q) if by_node else depth[b]
    logits = np.take_along_axis(logq, rows[:, :, None], 1) + r.normal(size=(B, Q, V)) / sharp
    x = torch.from_numpy(logits.astype(np.float32))
    if dtype == "bf16":
        x = x.bfloat16()
    return dict(logits=x, parent=torch.from_numpy(parent), tokens=torch.from_numpy(tokens),
                uniforms=torch.from_numpy(r.random((B, Q), np.float32)),
                temperature=torch.from_numpy(r.uniform(0.5, 1.5, B).astype(np.float32)),
                draft=torch.from_numpy(np.exp(logq).astype(np.float32)) if draft else None,
                by_node=by_node)


def outputs(B, Q):
    return [torch.full(s, -7, dtype=torch.int32, device="cuda")
            for s in ((B,), (B, Q), (B, Q))]


def call(s, out=None, **kw):
    B, Q, _ = s["logits"].shape
    out = out or outputs(B, Q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    tv.tree_sample(dev["logits"], dev["parent"], dev["tokens"], dev["uniforms"], *out,
                   temperature=dev["temperature"], draft_probs=dev["draft"],
                   draft_mode=tv.DRAFT_BY_NODE if s["by_node"] else tv.DRAFT_BY_DEPTH,
                   status=status, **kw)
    torch.cuda.synchronize()
    return [t.cpu().numpy() for t in out], int(status.item())


def expect(s):
    B, Q, V = s["logits"].shape
    x = s["logits"].double().numpy()
    res = [sm.sample_tree(x[b], s["parent"][b].numpy(), s["tokens"][b].numpy(),
                          s["uniforms"][b].numpy(),
                          1.0 if s["temperature"] is None else float(s["temperature"][b]),
                          None if s["draft"] is None else s["draft"][b].double().numpy(),
                          s["by_node"]) for b in range(B)]
    return [np.array([r[0] for r in res]), np.stack([r[1] for r in res]),
            np.stack([r[2] for r in res])]


def check(s, status=0):
    got, st = call(s)
    assert st == status
    for g, e in zip(got, expect(s)):
        assert np.array_equal(g, e)
    return got


@pytest.mark.parametrize("draft", [None, "depth", "node"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("B,Q,V", [(1, 1, 1), (1, 1, 7), (3, 9, 13), (5, 33, 1000),
                                   (2, 64, 4099), (1, 9, 32000), (4, 17, 50257),
                                   (40, 5, 2049), (200, 3, 517)])
def test_equals_the_rule(B, Q, V, dtype, draft):
    """Clusters of 1 to 16 CTAs, vocabularies that are no whole vectors, every form."""
    if V < 8 and Q > 1 and draft:
        pytest.skip("too few tokens to draw from")
    check(make(B * 1000 + Q + V, B, Q, V, dtype, draft))


@pytest.mark.parametrize("draft", [None, "depth", "node"])
def test_deep_walks(draft):
    """A chain whose tests all have the number zero is accepted whole."""
    s = make(4, 5, 40, 900, "bf16", draft, wide=1)
    s["uniforms"][:, 1:] = 0.0
    assert check(s)[0].min() == 39


def test_full_vocabulary():
    s = make(5, 2, 9, 163840, "fp32", "depth")
    check(s)
    check(dict(s, draft=None))


def test_largest_vocabulary_flat():
    """2^18 equal logits: the sum of the weights is as large as it gets."""
    s = make(6, 1, 2, 16)
    s["logits"] = torch.zeros((1, 2, 1 << 18))
    for u in (0.0, 0.25, 0.7310585975646973, 1 - 2.0 ** -24):
        s["uniforms"] = torch.tensor([[u, 0.999]])
        check(s)


@pytest.mark.parametrize("draft", [None, "depth"])
def test_many_rejections(draft):
    """A star of 63 children that the target hardly wants: every test and residual runs."""
    r = np.random.default_rng(8)
    s = make(9, 4, 64, 300, draft=draft)
    s["parent"][:, 1:] = 0
    for b in range(4):
        s["tokens"][b, 1:] = torch.from_numpy(r.permutation(300)[:63].astype(np.int32))
    s["uniforms"][:, 1:] = 1 - 2.0 ** -20
    a = check(s)[0]
    assert a.max() <= 1


def test_greedy_equals_tree_accept():
    s = make(10, 6, 21, 3001, "bf16")
    s["temperature"] = torch.zeros(6)
    x = s["logits"].cuda()
    x[:, :, 77] = x.amax(-1)  # a tie: the smaller index wins
    s["logits"] = x.cpu()
    got, st = call(s)
    a, path, emit = outputs(6, 21)
    tv.tree_accept(x, s["parent"].cuda(), s["tokens"].cuda(), a, path, emit)
    torch.cuda.synchronize()
    assert st == 0
    for g, e in zip(got, (a, path, emit)):
        assert np.array_equal(g, e.cpu().numpy())


def test_greedy_and_sampled_rows_mix():
    s = make(11, 8, 12, 700, draft="depth")
    s["temperature"][::3] = 0.0
    check(s)
    s["temperature"] = None
    check(s)


@pytest.mark.parametrize("T", [1e-38, 1e-4, 50.0, float("inf")])
def test_extreme_temperatures(T):
    """Nearly greedy, nearly uniform; masked tokens stay masked at any temperature."""
    s = make(12, 3, 7, 400)
    s["logits"][:, :, 100:] = float("-inf")
    s["temperature"] = torch.full((3,), T)
    if T == 1e-38:  # below the smallest scale: the maximum alone
        s["temperature"] = torch.zeros(3)
        e = expect(s)
        s["temperature"] = torch.full((3,), T)
        got, st = call(s)
        assert st == 0 and all(np.array_equal(g, x) for g, x in zip(got, e))
    elif T == float("inf"):
        s["temperature"] = torch.full((3,), 1e30)
        e = expect(s)
        s["temperature"] = torch.full((3,), T)
        got, st = call(s)
        assert st == 0 and all(np.array_equal(g, x) for g, x in zip(got, e))
    else:
        check(s)


def test_masks():
    """-inf masks: one token left, masked children, the lowest finite value."""
    s = make(13, 4, 8, 600)
    s["logits"][0, :, :] = float("-inf")
    s["logits"][0, :, 599] = -3.0
    s["logits"][1, :, s["tokens"][1].long()] = float("-inf")
    s["logits"][2] = torch.finfo(torch.float32).min
    s["logits"][2, :, 5] = 0.0
    s["logits"][3] = torch.finfo(torch.float32).min  # all equal: uniform
    got = check(s)
    assert got[2][0, 0] == 599


@pytest.mark.parametrize("what", ["nan", "inf", "masked"])
@pytest.mark.parametrize("T", [0.0, 1.0])
def test_rows_without_a_distribution(what, T):
    """The walk ends there without a bonus token; other sequences are untouched."""
    s = make(14, 3, 6, 5000)
    s["temperature"] = torch.full((3,), T)
    if what == "masked":
        s["logits"][1, 0] = float("-inf")
    else:
        s["logits"][1, 0, 4321] = float(what)
    got = check(s, tv.TV_ERR_INVALID_ARG)
    assert got[0][1] == 0 and got[2][1, 0] == -1


def test_bad_trees_temperatures_tokens_and_depths():
    s = make(15, 4, 6, 50, draft="depth")
    s["parent"][2, 3] = 4
    got, st = call(s)
    assert st == tv.TV_ERR_INVALID_TREE
    assert got[0][2] == 0 and got[1][2].tolist() == [0] + [-1] * 5
    assert (got[2][2] == -1).all()
    s = make(15, 4, 6, 50, draft="depth")
    e = expect(s)
    for bad in (-1.0, float("nan")):
        s["temperature"][1] = bad
        got, st = call(s)
        assert st == tv.TV_ERR_INVALID_ARG
        assert (got[2][1] == -1).all() and got[0][1] == 0
        for b in (0, 2, 3):
            assert got[0][b] == e[0][b] and np.array_equal(got[2][b], e[2][b])
    s = make(15, 4, 6, 50, draft="depth")
    s["tokens"][:, 1] = 50                          # outside the vocabulary: not tested
    s["tokens"][:, 2] = -1
    check(s)
    s = make(16, 4, 6, 50, draft="depth")
    s["parent"][:, 1:] = torch.arange(5, dtype=torch.int32)
    s["draft"] = s["draft"][:, :1]                  # one depth only
    s["uniforms"][:, 1] = 0.0                       # the first child is accepted
    got = check(s, tv.TV_ERR_BOUNDS)
    assert (got[0] == 1).all()


def test_uniforms_are_clamped():
    s = make(17, 4, 5, 64)
    for raw, used in ((-1.0, 0.0), (float("nan"), 0.0), (1.0, 1 - 2.0 ** -24),
                      (float("inf"), 1 - 2.0 ** -24)):
        s["uniforms"] = torch.full((4, 5), used)
        e = expect(s)
        s["uniforms"] = torch.full((4, 5), raw)
        got, _ = call(s)
        assert all(np.array_equal(g, x) for g, x in zip(got, e))


def test_equal_target_and_drafter():
    """p = g accepts the first child whatever its number; repeated sibling tokens."""
    s = make(18, 6, 9, 256, draft="node", sharp=1e30)
    s["temperature"] = None
    s["uniforms"][:, 1:] = 0.999
    check(s)
    s["tokens"][:, 2:] = s["tokens"][:, 1:2]
    check(s)
    check(dict(s, draft=None))


def test_strided_and_unaligned_rows():
    s = make(19, 3, 5, 1001, "bf16", draft="depth")
    e = expect(s)
    wide = torch.full((3 * 5, 1013), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:1004] = s["logits"].cuda().view(15, 1001)
    x = wide[:, 3:1004].unflatten(0, (3, 5))
    d = torch.full((3 * 5, 1009), float("nan"), device="cuda")
    d[:, 1:1002] = s["draft"].cuda().view(15, 1001)
    got, st = call(dict(s, logits=x, draft=d[:, 1:1002].unflatten(0, (3, 5))))
    assert st == 0 and all(np.array_equal(g, v) for g, v in zip(got, e))


def test_first_nodes_of_longer_rows():
    """One node per sequence, out of a tensor with more: rows a whole sequence apart."""
    s = make(23, 4, 6, 333, draft="depth")
    one = {k: v[:, :1] if isinstance(v, torch.Tensor) and v.dim() > 1 else v
           for k, v in s.items()}
    e = expect({k: v.contiguous() if isinstance(v, torch.Tensor) else v for k, v in one.items()})
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    out = outputs(4, 1)
    tv.tree_sample(dev["logits"][:, :1], dev["parent"][:, :1].contiguous(),
                   dev["tokens"][:, :1].contiguous(), dev["uniforms"][:, :1].contiguous(), *out,
                   temperature=dev["temperature"], draft_probs=dev["draft"][:, :1])
    torch.cuda.synchronize()
    assert all(np.array_equal(t.cpu().numpy(), x) for t, x in zip(out, e))


def test_captured_and_replayed_with_new_inputs():
    a, b = make(20, 4, 9, 3000, draft="depth"), make(21, 4, 9, 3000, draft="depth")
    dev = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    out = outputs(4, 9)

    def go():
        tv.tree_sample(dev["logits"], dev["parent"], dev["tokens"], dev["uniforms"], *out,
                       temperature=dev["temperature"], draft_probs=dev["draft"])

    go()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for s in (b, a):
        for k, v in s.items():
            if isinstance(v, torch.Tensor):
                dev[k].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(t.cpu().numpy(), e) for t, e in zip(out, expect(s)))


def test_two_streams_at_once():
    s = [make(22 + i, 8, 9, 20000) for i in range(2)]
    dev = [{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in s]
    out = [outputs(8, 9) for _ in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, o, st in zip(dev, out, streams):
            tv.tree_sample(d["logits"], d["parent"], d["tokens"], d["uniforms"], *o,
                           temperature=d["temperature"], stream=st)
    torch.cuda.synchronize()
    for x, o in zip(s, out):
        assert all(np.array_equal(t.cpu().numpy(), e) for t, e in zip(o, expect(x)))


def test_frequencies_follow_the_target():
    """4096 sequences with one tree and their own numbers: the first emitted token's counts
    against the target's probabilities (each within 5 standard deviations)."""
    one = make(30, 1, 4, 8, draft="depth", spread=1.0, sharp=1.0)
    B = 4096
    g = one["draft"][0, 0].double()
    r = np.random.default_rng(31)
    s = {k: (v.expand(B, *v.shape[1:]).contiguous() if isinstance(v, torch.Tensor) else v)
         for k, v in one.items()}
    s["parent"] = torch.tensor([[-1, 0, 0, 0]], dtype=torch.int32).expand(B, 4).contiguous()
    order = np.argsort(-(np.log(g.numpy()) + r.gumbel(size=(B, 8))), 1)[:, :3]
    s["tokens"] = torch.from_numpy(np.concatenate([np.zeros((B, 1)), order], 1).astype(np.int32))
    s["uniforms"] = torch.from_numpy(r.random((B, 4), np.float32))
    s["temperature"] = None
    got, _ = call(s)
    p = torch.softmax(one["logits"][0, 0].double(), -1).numpy()
    n = np.bincount(got[2][:, 0], minlength=8)
    assert (np.abs(n - B * p) <= 5 * np.sqrt(B * p * (1 - p))).all(), (n, B * p)
