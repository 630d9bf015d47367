"""GPU tests of the serving calls next to an attention call whose preparation may overlap the
call before it (overlap_prev), and inside captured graphs.

Each kernel of a pool or sampling call waits for the one before it and only then lets the next
start, so the preparation overlaps the call just before it and nothing earlier."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]

B, Q, H, DL, DR, PS, MOST, V = 24, 9, 64, 512, 64, 64, 12, 900
SCALE = 192 ** -0.5


def i32(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


class Batch:
    """Rows of one to ten pages over a pool with every cache row filled, and a causal attention
    call over what the rows hold and the Q keys behind it."""

    def __init__(self, seed):
        r = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape, s=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * s).bfloat16()

        # whole pages, so that the keys written next need a page that no table names yet
        self.length = PS * r.integers(1, 11, B)
        have = self.length // PS
        num = int(have.sum()) + 5 * B + 20000     # (many counts to scan: reserve takes longer)
        perm = r.permutation(num)
        table, ref, at = np.full((B, MOST), -1), np.zeros(num), 0
        for b in range(B):
            table[b, :have[b]] = perm[at:at + have[b]]
            ref[perm[at:at + have[b]]] = 1
            at += have[b]
        self.before = [i32(ref), i32(table), i32(have)]
        self.ref, self.table, self.n = (t.clone() for t in self.before)
        self.pool = tv.make_page_pool(self.ref, self.table, self.n, PS)
        self.c_kv, self.k_pe = randn(num * PS, DL), randn(num * PS, DR)
        self.ql, self.qr = randn(B, Q, H, DL, s=0.3), randn(B, Q, H, DR, s=0.3)
        self.len, self.new = i32(self.length), i32(self.length + Q)
        self.copies = torch.zeros((B, 3), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.anc = torch.full((B, Q), (1 << Q) - 1, dtype=torch.int64, device="cuda")
        self.out = torch.zeros((B, Q, H, DL), device="cuda")
        self.lse = torch.zeros((B, Q, H), device="cuda")

    def restore(self):
        for t, e in zip((self.ref, self.table, self.n), self.before):
            t.copy_(e)
        torch.cuda.synchronize()

    def reserve(self):
        tv.pages_reserve(self.pool, self.len, self.new, self.copies, status=self.status)

    def copy(self):
        tv.pages_copy(self.c_kv, self.k_pe, PS, self.copies, status=self.status)

    def attend(self, overlap, prefix=None, workspace=None):
        tv.verify_attn(self.ql, self.qr, self.c_kv, self.k_pe, self.len if prefix is None else prefix,
                       self.anc, self.out, self.lse, SCALE, 10 * PS, page_table=self.table,
                       status=self.status, overlap_prev=overlap, workspace=workspace,
                       path=tv.PATH_TCGEN05)


@pytest.fixture(scope="module")
def batch():
    return Batch(1)


def test_reserve_then_copy_then_overlapped_attention(batch):
    """The preparation may overlap the copy, not the reservation that wrote the tables."""
    s = batch
    s.restore()
    s.reserve()
    s.copy()
    torch.cuda.synchronize()
    s.attend(0)
    torch.cuda.synchronize()
    out, lse = s.out.clone(), s.lse.clone()
    assert int(s.status.item()) == 0 and torch.isfinite(out).all()
    for _ in range(20):
        s.restore()
        s.out.zero_()
        s.reserve()
        s.copy()
        s.attend(1)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        assert torch.equal(s.out, out) and torch.equal(s.lse, lse)


def test_sampling_between_reserve_and_overlapped_attention(batch):
    s = batch
    s.restore()
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn((B, Q, V), generator=g, device="cuda")
    parent = i32(np.tile(np.arange(-1, Q - 1), (B, 1)))
    tokens = torch.randint(0, V, (B, Q), generator=g, device="cuda", dtype=torch.int32)
    uni = torch.rand((B, Q), generator=g, device="cuda")
    acc, path, emit = (torch.empty(x, dtype=torch.int32, device="cuda")
                       for x in ((B,), (B, Q), (B, Q)))
    s.reserve()
    torch.cuda.synchronize()
    s.attend(0)
    torch.cuda.synchronize()
    out = s.out.clone()
    for _ in range(10):
        s.restore()
        s.out.zero_()
        s.reserve()
        tv.tree_sample(logits, parent, tokens, uni, acc, path, emit, status=s.status)
        s.attend(1)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0 and torch.equal(s.out, out)


def test_prompts_and_overlapped_attention_share_a_workspace(batch):
    """A workspace is free once the call's work on the stream is done: the next call's
    preparation must not write to it while the prompts' attention still reads it."""
    s = batch
    s.restore()
    s.reserve()
    torch.cuda.synchronize()
    T, H2 = 700, 64                                 # more items than SMs: no join at the end
    g = torch.Generator(device="cuda").manual_seed(6)

    def randn(*shape, k=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * k).bfloat16()

    q, qp, w = randn(T, H2, 128), randn(T, H2, 64), randn(H2, 256, DL, k=DL ** -0.5)
    start, pre = i32([0, 300, 700]), i32([0, 0])
    keys = randn(20 * PS, DL), randn(20 * PS, DR)
    pages = i32(np.arange(24).reshape(2, 12) % 20)
    out = torch.zeros((T, H2, 128), dtype=torch.bfloat16, device="cuda")
    args = tv.prefill_args(q, qp, w, *keys, start, pre, out, SCALE, 400, 400, 700, pages)
    need = max(tv.prefill_workspace_size(args),
               tv.workspace_size(tv.attn_args(s.ql, s.qr, s.c_kv, s.k_pe, s.len, s.anc, s.out,
                                              s.lse, SCALE, 10 * PS, s.table)))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def both(overlap):
        tv.prefill_attn(q, qp, w, *keys, start, pre, out, SCALE, 400, 400, 700, page_table=pages,
                        status=s.status, workspace=ws)
        if not overlap:
            torch.cuda.synchronize()
        s.attend(overlap, workspace=ws)
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        return out.clone(), s.out.clone()

    want = both(0)
    for _ in range(10):
        out.zero_()
        s.out.zero_()
        assert all(torch.equal(a, b) for a, b in zip(both(1), want))


def sampling(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return dict(logits=torch.randn((B, Q, V), generator=g, device="cuda"),
                parent=i32(np.tile(np.arange(-1, Q - 1), (B, 1))),
                tokens=torch.randint(0, V, (B, Q), generator=g, device="cuda", dtype=torch.int32),
                uniforms=torch.rand((B, Q), generator=g, device="cuda"),
                out=[torch.zeros(x, dtype=torch.int32, device="cuda") for x in ((B,), (B, Q), (B, Q))])


def sample(d, status, **kw):
    tv.tree_sample(d["logits"], d["parent"], d["tokens"], d["uniforms"], *d["out"], status=status,
                   **kw)


@pytest.mark.parametrize("branch", [False, True])
def test_captured_behind_copies_fills_and_another_stream(batch, branch):
    """In a graph the calls' kernels come first in it, behind memory copies and fills, and behind
    the join of a second stream that samples; replayed, they give what eager calls give."""
    s, d, e = batch, sampling(7), sampling(8)

    def go():
        main = torch.cuda.current_stream()
        if branch:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                sample(e, s.status)
        for t, v in zip((s.ref, s.table, s.n), s.before):
            t.copy_(v)
        s.reserve()
        s.copies_seen.copy_(s.copies)
        s.copy()
        d["out"][0].zero_()
        sample(d, s.status)
        if branch:
            main.wait_stream(side)
        s.attend(0)
        s.release_all.fill_(0)
        tv.pages_release(s.pool, s.release_all, status=s.status)

    s.copies_seen, s.release_all = torch.zeros_like(s.copies), torch.zeros_like(s.n)
    side = torch.cuda.Stream()
    go()
    torch.cuda.synchronize()
    seen = (s.ref, s.table, s.n, s.copies_seen, s.out, s.lse, *d["out"], *e["out"])
    want = [t.clone() for t in seen]
    assert int(s.status.item()) == 0 and int(s.ref.sum()) == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for _ in range(3):
        for t in (s.out, s.lse, *d["out"], *e["out"]):
            t.fill_(-3)
        g.replay()
        torch.cuda.synchronize()
        assert int(s.status.item()) == 0
        assert all(torch.equal(a, b) for a, b in zip(seen[:-3], want))
        if branch:
            assert all(torch.equal(a, b) for a, b in zip(e["out"], want[-3:]))
