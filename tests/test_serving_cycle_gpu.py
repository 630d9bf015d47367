"""The serving operators together, as a server runs them: a prompt's prefill over a paged
cache, forks of it, and verify cycles (reserve, copy on write, prologue, attention, sampled
acceptance, compaction, release) whose cache and tokens are followed by a plain model that
knows sequences as lists of rows."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import serving_model as sm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]

ROWS, Q, H, DL, DR, PS, PAGES, MOST, V = 5, 9, 8, 512, 64, 64, 40, 8, 701


def i32(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def test_prompt_fork_and_verify_cycles():
    r, g = np.random.default_rng(1), torch.Generator(device="cuda").manual_seed(1)

    def randn(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).bfloat16()

    table = torch.full((ROWS, MOST), -1, dtype=torch.int32, device="cuda")
    n_pages = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
    ref = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    pool = tv.make_page_pool(ref, table, n_pages, PS)
    copies = torch.zeros((ROWS, 3), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c_kv, k_pe = randn(PAGES * PS, DL), randn(PAGES * PS, DR)
    cache = tv.make_cache(table, PS, num_rows=PAGES * PS)

    def rows_of(row, n):
        t = table.cpu().numpy()[row]
        j = np.arange(n)
        return torch.from_numpy(t[j // PS].astype(np.int64) * PS + j % PS)

    # ---- the prompt ----
    n0 = 141
    length = np.zeros(ROWS, np.int64)
    tv.pages_reserve(pool, i32(length), i32([n0, 0, 0, 0, 0]), copies, status=status)
    length[0] = n0
    prompt = (randn(n0, DL), randn(n0, DR))
    at = rows_of(0, n0).cuda()
    c_kv[at], k_pe[at] = prompt
    q_nope, q_pe = randn(n0, H, 128), randn(n0, H, DR)
    w_kv, out = randn(H, 256, DL, s=DL ** -0.5), torch.zeros((n0, H, 128), device="cuda").bfloat16()
    tv.prefill_attn(q_nope, q_pe, w_kv, c_kv, k_pe, i32([0, n0]), i32([0]), out, 192 ** -0.5,
                    max_q_len=n0, max_kv_len=n0, total_kv=n0, page_table=table[:1].contiguous(),
                    status=status)
    e = sm.prefill(f64(q_nope), f64(q_pe), f64(w_kv), f64(prompt[0]), f64(prompt[1]), 0,
                   192 ** -0.5)
    rms = np.sqrt(((f64(out) - e) ** 2).mean(-1)) / np.sqrt((e ** 2).mean(-1))
    assert rms.max() <= 2.0 ** -7

    # ---- three samples fork from it; row 3 stays free ----
    tv.pages_fork(pool, i32([-1, 0, 0, -1, 0]), i32([0, n0, n0, 0, n0]), status=status)
    length[[1, 2, 4]] = n0
    live = np.array([0, 1, 2, 4])
    logical = {b: [prompt[0].clone(), prompt[1].clone()] for b in live}
    said = {b: [] for b in live}

    for step in range(6):
        parent = np.full((ROWS, Q), -1, np.int32)
        for b in range(ROWS):
            parent[b, 1:] = [r.integers(max(0, i - 3), i) for i in range(1, Q)]
        new = np.where(np.isin(np.arange(ROWS), live), length + Q, -1)
        tv.pages_reserve(pool, i32(length), i32(new), copies, status=status)
        tv.pages_copy(c_kv, k_pe, PS, copies, status=status)
        # the verify kernels take the live rows
        sub = table[torch.from_numpy(live).cuda()].contiguous()
        sub_cache = tv.make_cache(sub, PS, num_rows=PAGES * PS)
        par, pre = i32(parent[live]), i32(length[live])
        B = len(live)
        ckv_tree, kpe_tree = randn(B, Q, DL), randn(B, Q, DR)
        ql, qr = randn(B, Q, H, DL, s=192 ** -0.5), randn(B, Q, H, DR, s=192 ** -0.5)
        anc = torch.empty((B, Q), dtype=torch.int64, device="cuda")
        depth = torch.empty((B, Q), dtype=torch.int32, device="cuda")
        tv.verify_prologue(par, pre, qr, qr, kpe_tree, ckv_tree, c_kv, k_pe, sub_cache, anc, depth,
                           status=status)
        o = torch.empty((B, Q, H, DL), device="cuda")
        lse = torch.empty((B, Q, H), device="cuda")
        tv.verify_attn(ql, qr, c_kv, k_pe, pre, anc, o, lse, 192 ** -0.5, int(length.max()),
                       page_table=sub, status=status)
        # row 0's first node against float64 over the model's own rows
        keys = [torch.cat([logical[live[0]][k], x]) for k, x in
                ((0, ckv_tree[0, :1]), (1, k_pe[rows_of(live[0], length[live[0]] + 1)[-1:].cuda()]))]
        s = (f64(ql[0, 0]) @ f64(keys[0]).T + f64(qr[0, 0]) @ f64(keys[1]).T) * 192 ** -0.5
        p = np.exp(s - s.max(-1, keepdims=True))
        e = (p / p.sum(-1, keepdims=True)) @ f64(keys[0])
        rms = np.sqrt(((f64(o[0, 0]) - e) ** 2).mean(-1)) / np.sqrt((e ** 2).mean(-1))
        assert rms.max() <= 2.0 ** -7
        # sampled acceptance, its rows moved together, the pages behind them given back
        draft = torch.softmax(3 * torch.randn((B, Q, V), generator=g, device="cuda"), -1)
        logits = torch.log(draft) + 0.5 * torch.randn((B, Q, V), generator=g, device="cuda")
        order = torch.multinomial(draft.view(-1, V), Q, generator=g).view(B, Q, Q).cpu().numpy()
        tokens, taken = np.zeros((B, Q), np.int32), np.zeros((B, Q), np.int64)
        for b in range(B):
            for i in range(1, Q):
                n = parent[live[b], i]
                tokens[b, i] = order[b, n, taken[b, n]]
                taken[b, n] += 1
        uni = torch.rand((B, Q), generator=g, device="cuda")
        acc, path, emit = (torch.empty(s, dtype=torch.int32, device="cuda")
                           for s in ((B,), (B, Q), (B, Q)))
        tv.tree_sample(logits, par, i32(tokens), uni, acc, path, emit, draft_probs=draft,
                       draft_mode=tv.DRAFT_BY_NODE, status=status)
        moved = torch.empty(B, dtype=torch.int32, device="cuda")
        kpe_rot = {b: k_pe[rows_of(live[b], length[live[b]] + Q)[-Q:].cuda()].clone()
                   for b in range(B)}
        tv.compact_kv(c_kv, k_pe, sub_cache, pre, path, acc, moved, status=status)
        for b in range(B):
            a, pth, new_tokens = sm.sample_tree(f64(logits[b]), parent[live[b]], tokens[b],
                                                uni[b].cpu().numpy(), 1.0, f64(draft[b]), True)
            assert a == int(acc[b]) and np.array_equal(pth, path[b].cpu().numpy())
            assert np.array_equal(new_tokens, emit[b].cpu().numpy())
            said[live[b]] += new_tokens[:a + 1].tolist()
            kept = torch.from_numpy(pth[:a + 1].astype(np.int64)).cuda()
            logical[live[b]][0] = torch.cat([logical[live[b]][0], ckv_tree[b][kept]])
            logical[live[b]][1] = torch.cat([logical[live[b]][1], kpe_rot[b][kept]])
            length[live[b]] += a + 1
        assert np.array_equal(moved.cpu().numpy(), length[live])
        keep = np.full(ROWS, -1)
        keep[live] = length[live]
        if step == 3:  # a sample ends, another forks from a living one in the middle of a page
            keep[2] = 0
        tv.pages_release(pool, i32(keep), status=status)
        if step == 3:
            cut = int(length[4]) - 3
            tv.pages_fork(pool, i32([-1, -1, 4, -1, -1]), i32([0, 0, cut, 0, 0]), status=status)
            logical[2] = [t[:cut].clone() for t in logical[4]]
            said[2] = None
            length[2] = cut
            moves = torch.empty((PAGES, 3), dtype=torch.int32, device="cuda")
            n_moves = torch.empty(1, dtype=torch.int32, device="cuda")
            tv.pages_compact(pool, moves, n_moves, status=status)
            tv.pages_copy(c_kv, k_pe, PS, moves, count=n_moves, status=status)
            assert (ref > 0).sum() == (ref[:int((ref > 0).sum())] > 0).sum()
        if said[2] is None:
            said[2] = []
        # every sequence reads back as the model has it
        for b in live:
            at = rows_of(b, length[b]).cuda()
            assert torch.equal(c_kv[at], logical[b][0]) and torch.equal(k_pe[at], logical[b][1])
        count = np.zeros(PAGES, np.int64)
        t, n = table.cpu().numpy(), n_pages.cpu().numpy()
        for b in range(ROWS):
            np.add.at(count, t[b, :n[b]], 1)
        assert np.array_equal(count, ref.cpu().numpy())
    assert int(status.item()) == 0
    assert sum(len(x) for x in said.values()) >= 6 * 4
