"""The decode cycle's operators together, as a server runs them for samples of one prompt: the
prompt's rows normed, rotated and appended (tv_norm_rope), forks of it, and steps of one token a
sample (reserve, copy on write, tv_norm_rope, tv_shared_attn, tv_token_sample), the whole step
captured once and replayed, followed by a plain model that knows sequences as lists of rows."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import decode_model as dm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]

N, H, DL, DR, PS, PAGES, MOST, V = 7, 16, 512, 64, 64, 60, 16, 5003
SCALE, LAYOUT = 192 ** -0.5, tv.ROPE_INTERLEAVED


def i32(v):
    return torch.from_numpy(np.ascontiguousarray(v, np.int32)).cuda()


def f64(t):
    return t.double().cpu().numpy()


def test_samples_of_one_prompt():
    g = torch.Generator(device="cuda").manual_seed(3)

    def randn(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).bfloat16()

    table = torch.full((N, MOST), -1, dtype=torch.int32, device="cuda")
    n_pages = torch.zeros(N, dtype=torch.int32, device="cuda")
    ref = torch.zeros(PAGES, dtype=torch.int32, device="cuda")
    pool = tv.make_page_pool(ref, table, n_pages, PS)
    copies = torch.zeros((N, 3), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c_kv = torch.full((PAGES * PS, DL), float("nan"), device="cuda").bfloat16()
    k_pe = torch.full((PAGES * PS, DR), float("nan"), device="cuda").bfloat16()
    weight = (1 + 0.2 * randn(DL)).bfloat16()
    scaling = tv.rope_scaling(kind=tv.ROPE_YARN, factor=8.0, original_context=512)
    f, mag = dm.frequencies(DR, kind="yarn", factor=8.0, context=512.0), \
        dm.magnitude("yarn", 8.0)

    def rows_of(row, n):
        t = table.cpu().numpy()[row]
        j = np.arange(n)
        return torch.from_numpy(t[j // PS].astype(np.int64) * PS + j % PS).cuda()

    def model_rows(kv, at):
        """The cache rows of projected keys kv [n, DL+DR] at positions at, in 64 bits."""
        x = f64(kv)
        c = dm.norm(x[:, :DL], f64(weight), 1e-6)
        return c, dm.turn(x[:, None, DL:], at[:, None] * f[None], "pairs", mag)[:, 0]

    # ---- the prompt's rows, in one call ----
    n0 = 700
    tv.pages_reserve(pool, i32([0] * N), i32([n0] + [0] * (N - 1)), copies, status=status)
    prompt = randn(n0, DL + DR)
    tv.norm_rope(None, prompt, i32([0, n0]), i32([0]), None, None, c_kv, k_pe, kv_weight=weight,
                 layout=LAYOUT, scaling=scaling, page_table=table[:1].contiguous(), status=status)
    c_ref, k_ref = model_rows(prompt, np.arange(n0))
    at = rows_of(0, n0)
    for got, want in ((c_kv[at], c_ref), (k_pe[at], k_ref)):
        assert np.abs(f64(got) - want).max() <= 2.0 ** -7 * np.abs(want).max()
    # what the cache holds from here on is the model's too
    logical = [[c_kv[at].clone(), k_pe[at].clone()] for _ in range(N)]

    # ---- samples fork from it ----
    tv.pages_fork(pool, i32([-1] + [0] * (N - 1)), i32([0] + [n0] * (N - 1)), status=status)

    # ---- one step, captured: its inputs and lengths are read from these ----
    length, grown = i32([n0] * N), i32([n0 + 1] * N)
    q_pe_in, kv = randn(N, H, DR), randn(N, DL + DR)
    q_latent, q_pe = randn(N, 1, H, DL, s=0.3), torch.zeros((N, H, DR), device="cuda").bfloat16()
    out = torch.zeros((N, 1, H, DL), device="cuda")
    lse = torch.zeros((N, 1, H), device="cuda")
    logits, uni = torch.randn((N, V), generator=g, device="cuda"), torch.rand(N, device="cuda")
    tokens, kept = i32([0] * N), i32([0] * N)
    temp = torch.full((N,), 0.8, device="cuda")
    top_k, top_p = i32([50] * N), torch.full((N,), 0.9, device="cuda")
    start, group, shared = i32(np.arange(N + 1)), i32([0, N]), i32([n0])

    def step():
        tv.pages_reserve(pool, length, grown, copies, status=status)
        tv.pages_copy(c_kv, k_pe, PS, copies, status=status)
        tv.norm_rope(q_pe_in, kv, start, length, None, q_pe, c_kv, k_pe, kv_weight=weight,
                     layout=LAYOUT, scaling=scaling, page_table=table, status=status)
        tv.shared_attn(q_latent, q_pe.view(N, 1, H, DR), c_kv, k_pe, length, group, shared, out,
                       lse, SCALE, max_prefix_len=(MOST * PS) - 1, page_table=table,
                       status=status)
        tv.token_sample(logits, uni, tokens, temperature=temp, top_k=top_k, top_p=top_p,
                        kept=kept, status=status)

    graph, said = None, [[] for _ in range(N)]
    for i in range(90):                      # past the next page's end
        q_pe_in.copy_(randn(N, H, DR))
        kv.copy_(randn(N, DL + DR))
        q_latent.copy_(randn(N, 1, H, DL, s=0.3))
        logits.copy_(3 * torch.randn((N, V), generator=g, device="cuda"))
        uni.copy_(torch.rand(N, generator=g, device="cuda"))
        if i == 0:
            step()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        n = n0 + i
        for b in range(N):
            row = rows_of(b, n + 1)[-1:]
            logical[b][0] = torch.cat([logical[b][0], c_kv[row]])
            logical[b][1] = torch.cat([logical[b][1], k_pe[row]])
            if i % 13 == 0:
                c_new, k_new = model_rows(kv[b:b + 1], np.array([n]))
                for got, want in ((c_kv[row], c_new), (k_pe[row], k_new)):
                    assert np.abs(f64(got) - want).max() <= 2.0 ** -7 * np.abs(want).max()
                z = dm.turn(f64(q_pe_in[b:b + 1]), np.full((1, 1), n) * f[None], "pairs", mag)
                assert np.abs(f64(q_pe[b:b + 1]) - z).max() <= 2.0 ** -7 * np.abs(z).max()
                seen = torch.ones((1, n + 1), dtype=torch.bool, device="cuda")
                e, l, _, _ = dm.attention(q_latent[b], q_pe[b][None], *logical[b], seen, SCALE)
                err = ((out[b].double() - e) ** 2).mean(-1).sqrt() / (e ** 2).mean(-1).sqrt()
                assert err.max() <= 2.0 ** -8
                assert (lse[b].double() - l).abs().max() <= 1e-4
        for b in range(N):
            want = dm.next_token(f64(logits[b]), float(uni[b]), 0.8, 50, 0.9)
            assert (int(tokens[b]), int(kept[b])) == want
            said[b].append(want[0])
        length += 1
        grown += 1
    assert int(status.item()) == 0
    # every sequence reads back as the model has it, and the prompt's whole pages are still one
    for b in range(N):
        at = rows_of(b, n0 + 90)
        assert torch.equal(c_kv[at], logical[b][0]) and torch.equal(k_pe[at], logical[b][1])
    t = table.cpu().numpy()
    assert (t[:, :n0 // PS] == t[0, :n0 // PS]).all()
    assert len(set(t[:, n0 // PS].tolist())) == N
    assert len({tuple(s) for s in said}) == N
