"""Measured calls of the serving operators around the paged latent cache.

Three operators, each in its plain form (elementary torch operations) and as a user's
program calls it in this package:

  sample   sampled acceptance of a verified draft tree from given uniform numbers
  pages    pages of the cache: fork, copy-on-write reserve and release; compaction
  prefill  causal attention of prompts over the latent cache in its expanded form

``own`` selects the form that ``run`` computes.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


def _tv():
    from speculative_decoding_tree_04_gb300 import tv
    return tv


def _ints(text):
    return [int(x) for x in text.split(",")]


def _text(values):
    return ",".join(str(int(v)) for v in values)


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def listed():
    return [
        # One user, a short draft tree over a 32000-token vocabulary: latency of one call.
        dict(name="sample_one", op="sample", B=1, Q=9, V=32000, dt="bf16", draft="none",
             temp=0.8),
        # The B32 Q33 verify workload with its 163840-token float32 logits; candidates
        # chosen by rank (the framework's tree builder), one temperature.
        dict(name="sample_b32", op="sample", B=32, Q=33, V=163840, dt="fp32", draft="none",
             temp=1.0),
        # The B8 Q9 verify workload, candidates drawn from a block drafter (one
        # distribution per depth); some sequences greedy, the others at temperature 0.7.
        dict(name="sample_draft_b8", op="sample", B=8, Q=9, V=163840, dt="bf16",
             draft="depth", temp=0.7),
        # A full batch with an autoregressive drafter (one distribution per node) and an
        # odd vocabulary, whose rows start at any alignment.
        dict(name="sample_draft_b64", op="sample", B=64, Q=17, V=50257, dt="fp32",
             draft="node", temp=1.0),
        # Parallel sampling of one prompt: 4 samples fork from it, every row reserves the
        # slots of its next draft tree.
        dict(name="fork_one", op="fork", parents=1, children=4, keys=700, spread=0, grow=9,
             page=64, layers=1, spare=16, DL=512, DR=64, dt="bf16"),
        # 64 prompts of up to 8192 tokens, 7 samples each, a cache of four layers.
        dict(name="fork_b64", op="fork", parents=64, children=7, keys=8150, spread=4000,
             grow=33, page=64, layers=4, spare=1024, DL=512, DR=64, dt="bf16"),
        # A small float32 cache, every second page in use.
        dict(name="compact_small", op="compact", rows=8, pages=512, used=200, page=16,
             layers=1, DL=128, DR=16, dt="fp32"),
        # A long-running server's cache before memory is handed back: 16384 pages of two
        # layers, 40 % in use all over it.
        dict(name="compact_large", op="compact", rows=96, pages=16384, used=6550, page=64,
             layers=2, DL=512, DR=64, dt="bf16"),
        # A short question: latency.
        dict(name="prefill_one", op="prefill", H=16, lens="33", prefixes="0", paged=True),
        # The 4096-token causal prefill of one prompt, 64 heads.
        dict(name="prefill_4096", op="prefill", H=64, lens="4096", prefixes="0", paged=False),
        # A ragged batch as a scheduler forms it: new prompts, chunks after a cached
        # prefix, and a single token.
        dict(name="prefill_ragged", op="prefill", H=64, lens="1,700,33,1500,257,128",
             prefixes="900,0,1777,512,64,3000", paged=True),
        # Chunks of 256 tokens far into long prompts, 16 heads.
        dict(name="prefill_chunks", op="prefill", H=16, lens="256,256,256,256",
             prefixes="6000,3840,2048,5111", paged=True),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["sample", "sample", "fork", "compact", "prefill", "prefill"])
    if op == "sample":
        B, V = _logint(rng, 1, 64), _logint(rng, 100, 163840)
        Q = min(rng.randint(1, 64), max(1, 32 * 33 * 163840 // (B * V)))
        return dict(op=op, B=B, Q=Q, V=V, dt=rng.choice(["bf16", "fp32"]),
                    draft=rng.choice(["none", "depth", "node"]),
                    temp=round(rng.uniform(0.4, 1.4), 2))
    if op == "fork":
        parents, children = _logint(rng, 1, 48), rng.randint(1, 7)
        keys = _logint(rng, 40, 6000)
        return dict(op=op, parents=parents, children=children, keys=keys,
                    spread=rng.randint(0, keys - 1), grow=rng.randint(1, 64),
                    page=rng.choice([16, 64]), layers=rng.randint(1, 3),
                    spare=rng.randint(0, 300),
                    DL=rng.choice([64, 128, 512]), DR=rng.choice([16, 64]),
                    dt=rng.choice(["bf16", "fp32"]))
    if op == "compact":
        pages = _logint(rng, 40, 8000)
        return dict(op=op, rows=_logint(rng, 1, 96), pages=pages,
                    used=max(1, int(pages * rng.uniform(0.1, 0.9))),
                    page=rng.choice([16, 64]), layers=rng.randint(1, 2),
                    DL=rng.choice([64, 128, 512]), DR=rng.choice([16, 64]),
                    dt=rng.choice(["bf16", "fp32"]))
    B = rng.randint(1, 6)
    return dict(op=op, H=rng.choice([1, 5, 8, 16, 64]),
                lens=_text(_logint(rng, 1, 1600) for _ in range(B)),
                prefixes=_text(rng.choice([0, _logint(rng, 1, 3000)]) for _ in range(B)),
                paged=rng.random() < 0.7)


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _torch_dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _sample_inputs(case, seed):
    """A draft tree, its tokens and the target's logits.

    The drafter's distribution over the vocabulary falls off with the rank of a token
    (weight rank^-2.2); the target's logits are the drafter's plus noise.  The children
    of a node are the drafter's best tokens (draft "none") or a draw of it without
    replacement, in the order drawn.
    """
    B, Q, V = case["B"], case["Q"], case["V"]
    r = np.random.default_rng([int(seed), 5])
    parent = np.full((B, Q), -1, np.int32)
    depth = np.zeros((B, Q), np.int64)
    rank = np.zeros((B, Q), np.int64)        # how many siblings come before node i
    for b in range(B):
        kids = np.zeros(Q, np.int64)
        for i in range(1, Q):
            # a node takes at most V children (a draw without replacement ends there)
            p = int(r.integers(max(0, i - 6), i))
            while kids[p] >= min(V, 16):
                p += 1
            parent[b, i], depth[b, i], rank[b, i] = p, depth[b, p] + 1, kids[p]
            kids[p] += 1
    g = _gen(seed)
    by_node = case["draft"] == "node"
    n_rows = Q if by_node else int(depth.max()) + 1
    # one drafter row per node or per depth of the parent
    u = torch.rand((B, n_rows, V), generator=g, device=DEV)
    logq = -2.2 * torch.log1p(u * V)
    del u
    logq -= torch.logsumexp(logq.double(), -1, keepdim=True).float()
    K = min(16, V)
    if case["draft"] == "none":
        score = logq
    else:  # Gumbel perturbation: the order of a draw without replacement
        e = torch.empty_like(logq).exponential_(generator=g).clamp_(min=1e-30)
        score = logq - torch.log(e)
    top = torch.topk(score, K, dim=-1).indices
    del score
    row_of = torch.from_numpy(np.broadcast_to(np.arange(Q), (B, Q)).copy()
                              if by_node else depth).to(DEV)
    par = torch.from_numpy(parent.astype(np.int64)).to(DEV).clamp_(min=0)
    par_row = torch.gather(row_of, 1, par)
    bi = torch.arange(B, device=DEV)[:, None]
    tokens = top[bi, par_row, torch.from_numpy(rank).to(DEV)]
    tokens[:, 0] = torch.randint(0, V, (B,), generator=g, device=DEV)
    logits = torch.empty((B, Q, V), dtype=_torch_dt(case["dt"]), device=DEV)
    for i in range(Q):
        x = logq[bi[:, 0], row_of[:, i]]
        x = x + 0.5 * torch.randn((B, V), generator=g, device=DEV)
        logits[:, i] = x.to(logits.dtype)
    temp = torch.full((B,), case["temp"], dtype=torch.float32, device=DEV)
    if case["draft"] == "depth":
        temp[::4] = 0.0                      # a mixed batch: every fourth row greedy
    probs = None
    if case["draft"] != "none":
        probs = logq.exp()
    return dict(logits=logits, parent=torch.from_numpy(parent).to(DEV),
                tokens=tokens.to(torch.int32), temp=temp, probs=probs, by_node=by_node,
                uniforms=torch.rand((B, Q), generator=g, device=DEV))


def _lengths(case):
    """Keys of each prompt of a fork case, spread evenly below the longest."""
    n = case["parents"]
    return [case["keys"] - (case["spread"] * i) // max(1, n - 1) if n > 1 else case["keys"]
            for i in range(n)]


def _cache(case, num_pages, g):
    rows, dt = num_pages * case["page"], _torch_dt(case["dt"])
    c = torch.randn((case["layers"], rows, case["DL"]), generator=g, device=DEV,
                    dtype=torch.float32).to(dt)
    k = torch.randn((case["layers"], rows, case["DR"]), generator=g, device=DEV,
                    dtype=torch.float32).to(dt)
    return c, k


def _fork_inputs(case, seed):
    ps, n, m = case["page"], case["parents"], case["children"]
    lens = _lengths(case)
    have = [-(-x // ps) for x in lens]
    rows = n * (1 + m)
    most = max(-(-(x + case["grow"]) // ps) for x in lens)
    # a page for each row's growth and copied page, and some spare ones
    num = sum(have) + sum((1 + m) * (-(-(x + case["grow"]) // ps) - x // ps)
                          for x in lens) + case["spare"]
    r = np.random.default_rng([int(seed), 6])
    perm = r.permutation(num)
    table = np.full((rows, most), -1, np.int32)
    ref = np.zeros(num, np.int32)
    n_pages = np.zeros(rows, np.int32)
    at = 0
    for i in range(n):
        table[i, :have[i]] = perm[at:at + have[i]]
        ref[perm[at:at + have[i]]] = 1
        n_pages[i] = have[i]
        at += have[i]
    source = np.full(rows, -1, np.int32)
    length = np.zeros(rows, np.int32)
    keep = np.full(rows, -1, np.int32)
    length[:n] = lens
    for j in range(n, rows):
        source[j] = (j - n) % n
        length[j] = lens[source[j]]
        keep[j] = 0
    return dict(table=table, ref=ref, n_pages=n_pages, source=source, length=length,
                keep=keep, new_length=length + case["grow"], num=num)


def _compact_inputs(case, seed):
    num, used, rows = case["pages"], case["used"], case["rows"]
    r = np.random.default_rng([int(seed), 7])
    mine = r.permutation(num)[:used]
    # rows of unequal length: the page counts grow with the square of the row's index
    cut = [used * i * i // (rows * rows) for i in range(1, rows)]
    parts = np.split(mine, cut)
    shared = mine[:min(3, used)]             # a prefix that every fourth row shares
    lists = [np.concatenate([shared, p]) if i % 4 == 1 else p for i, p in enumerate(parts)]
    most = max(1, max(len(p) for p in lists))
    table = np.full((rows, most), -1, np.int32)
    ref = np.zeros(num, np.int32)
    n_pages = np.zeros(rows, np.int32)
    for i, p in enumerate(lists):
        table[i, :len(p)] = p
        n_pages[i] = len(p)
        np.add.at(ref, p, 1)
    return dict(table=table, ref=ref, n_pages=n_pages, num=num)


def _prefill_inputs(case, seed):
    H, lens, pre = case["H"], _ints(case["lens"]), _ints(case["prefixes"])
    g = _gen(seed)
    T, B = sum(lens), len(lens)
    keys = [a + p for a, p in zip(lens, pre)]

    def randn(*shape, scale=1.0):
        x = torch.randn(shape, generator=g, device=DEV)
        return (x * scale).to(torch.bfloat16)

    page, table, stride = 64, None, 0
    if case["paged"]:
        need = [-(-k // page) for k in keys]
        r = np.random.default_rng([int(seed), 8])
        perm = r.permutation(sum(need) + 5)
        t = np.zeros((B, max(need)), np.int32)
        at = 0
        for b in range(B):
            t[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        table = torch.from_numpy(t).to(DEV)
        rows = len(perm) * page
    else:
        stride = max(keys)
        rows = B * stride
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return dict(q_nope=randn(T, H, 128), q_pe=randn(T, H, 64),
                w_kv=randn(H, 256, 512, scale=512 ** -0.5),
                c_kv=randn(rows, 512), k_pe=randn(rows, 64),
                q_start=torch.from_numpy(start).to(DEV),
                prefix_len=torch.tensor(pre, dtype=torch.int32, device=DEV),
                table=table, page=page, stride=stride, lens=lens, pre=pre, keys=keys,
                scale=192 ** -0.5)


def prepare(case, seed):
    op = case["op"]
    if op == "sample":
        s = _sample_inputs(case, seed)
        B, Q = case["B"], case["Q"]
        s["accept_len"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["path"] = torch.zeros((B, Q), dtype=torch.int32, device=DEV)
        s["new_tokens"] = torch.zeros((B, Q), dtype=torch.int32, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    elif op == "fork":
        h = _fork_inputs(case, seed)
        s = {k: torch.from_numpy(v).to(DEV) for k, v in h.items() if k != "num"}
        s["c_kv"], s["k_pe"] = _cache(case, h["num"], _gen(seed))
        s["copies"] = torch.full((len(h["length"]), 3), -1, dtype=torch.int32, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    elif op == "compact":
        h = _compact_inputs(case, seed)
        s = {k: torch.from_numpy(v).to(DEV) for k, v in h.items() if k != "num"}
        s["table0"], s["ref0"] = s["table"].clone(), s["ref"].clone()
        s["c_kv"], s["k_pe"] = _cache(case, h["num"], _gen(seed))
        s["moves"] = torch.full((h["num"], 3), -1, dtype=torch.int32, device=DEV)
        s["n_moves"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    else:
        s = _prefill_inputs(case, seed)
        s["out"] = torch.zeros((sum(s["lens"]), case["H"], 128), dtype=torch.bfloat16,
                               device=DEV)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    if op in ("fork", "compact") and own:
        s["pool"] = _tv().make_page_pool(s["ref"], s["table"], s["n_pages"], case["page"])
    s["case"] = case
    return s


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "sample":
        return _own_sample(s) if own else _plain_sample(s)
    if op == "fork":
        return _own_fork(s) if own else _plain_fork(s)
    if op == "compact":
        return _own_compact(s) if own else _plain_compact(s)
    return _own_prefill(s) if own else _plain_prefill(s)


def _own_sample(s):
    tv = _tv()
    tv.tree_sample(s["logits"], s["parent"], s["tokens"], s["uniforms"], s["accept_len"],
                   s["path"], s["new_tokens"], temperature=s["temp"], draft_probs=s["probs"],
                   draft_mode=tv.DRAFT_BY_NODE if s["by_node"] else tv.DRAFT_BY_DEPTH,
                   status=s["status"])
    return s["accept_len"], s["path"], s["new_tokens"]


def _own_fork(s):
    # the rows that end free their pages, new samples fork from the prompts, every row
    # gets the pages of its next draft tree, and shared last pages are copied
    tv = _tv()
    tv.pages_release(s["pool"], s["keep"], status=s["status"])
    tv.pages_fork(s["pool"], s["source"], s["length"], status=s["status"])
    tv.pages_reserve(s["pool"], s["length"], s["new_length"], s["copies"],
                     status=s["status"])
    tv.pages_copy(s["c_kv"], s["k_pe"], s["case"]["page"], s["copies"], status=s["status"])
    return s["table"], s["n_pages"], s["ref"], s["copies"], s["c_kv"], s["k_pe"]


def _own_compact(s):
    tv = _tv()
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    tv.pages_compact(s["pool"], s["moves"], s["n_moves"], status=s["status"])
    tv.pages_copy(s["c_kv"], s["k_pe"], s["case"]["page"], s["moves"], count=s["n_moves"],
                  status=s["status"])
    return s["table"], s["n_pages"], s["ref"], s["n_moves"], s["c_kv"], s["k_pe"]


def _own_prefill(s):
    _tv().prefill_attn(s["q_nope"], s["q_pe"], s["w_kv"], s["c_kv"], s["k_pe"],
                       s["q_start"], s["prefix_len"], s["out"], s["scale"],
                       max_q_len=max(s["lens"]), max_kv_len=max(s["keys"]),
                       total_kv=sum(s["keys"]), page_table=s["table"],
                       page_size=s["page"], kv_stride_b=s["stride"], status=s["status"])
    return s["out"]


def _plain_weights(logits, temp):
    """softmax(logits / temp) in 64 bits; the point mass of the first maximum at 0."""
    x = logits.double()
    t = temp.double()[:, None]
    y = x / torch.where(t > 0, t, torch.ones_like(t))
    w = torch.exp(y - y.max(-1, keepdim=True).values)
    w = w / w.sum(-1, keepdim=True)
    first = torch.zeros_like(w).scatter_(1, x.argmax(-1, keepdim=True), 1.0)
    return torch.where(t > 0, w, first)


def _plain_sample(s):
    # 64 bits: the drawn token turns on a running sum over the vocabulary
    logits, parent, tokens, u = s["logits"], s["parent"], s["tokens"].long(), s["uniforms"]
    B, Q, V = logits.shape
    bi = torch.arange(B, device=DEV)
    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    depth = torch.zeros(B, dtype=torch.long, device=DEV)
    path = torch.full((B, Q), -1, dtype=torch.int32, device=DEV)
    path[:, 0] = 0
    emit = torch.full((B, Q), -1, dtype=torch.int32, device=DEV)
    w = _plain_weights(logits[:, 0], s["temp"])
    drafts = s["probs"] is not None
    if drafts:
        g = s["probs"][:, 0].double()
        G = torch.ones(B, dtype=torch.float64, device=DEV)
    # a parent comes before its children, so one sweep over the nodes walks the tree
    for i in range(1, Q):
        on = parent[:, i] == cur
        x = tokens[:, i]
        wx, W = w[bi, x], w.sum(-1)
        ui = u[:, i].double()
        if drafts:
            gx = g[bi, x]
            on = on & (G > 0)
            ok = on & (ui * gx * W < wx * G)
        else:
            ok = on & (ui * W < wx)
        no = on & ~ok
        if drafts:
            left = (w - g * (W / G)[:, None]).clamp_(min=0)
            w = torch.where(no[:, None], left, w)
            G = torch.where(no, G - gx, G)
            g[bi, x] = torch.where(no, torch.zeros_like(gx), gx)
        w[bi, x] = torch.where(no, torch.zeros_like(wx), w[bi, x])
        cur = torch.where(ok, i, cur)
        emit[bi, depth] = torch.where(ok, x.int(), emit[bi, depth])
        depth = depth + ok.long()
        path[bi, depth] = torch.where(ok, i, path[bi, depth]).int()
        w = torch.where(ok[:, None], _plain_weights(logits[:, i], s["temp"]), w)
        if drafts:
            row = torch.full_like(depth, i) if s["by_node"] else depth
            row = row.clamp(max=s["probs"].shape[1] - 1)
            g = torch.where(ok[:, None], s["probs"][bi, row].double(), g)
            G = torch.where(ok, torch.ones_like(G), G)
    run_sum = torch.cumsum(w, -1)
    aim = u[:, 0].double() * run_sum[:, -1]
    drawn = (run_sum <= aim[:, None]).sum(-1).clamp(max=V - 1)
    emit[bi, depth] = drawn.int()
    return depth.int(), path, emit


def _plain_copy(s, copies):
    """Copy the first rows of page src to page dst, in every layer, for each (src, dst,
    rows) of the list."""
    ps = s["case"]["page"]
    c = copies.long()
    r = torch.arange(ps, device=DEV)[None]
    on = (c[:, :1] >= 0) & (r < c[:, 2:])
    src, dst = (c[:, :1] * ps + r)[on], (c[:, 1:2] * ps + r)[on]
    for t in (s["c_kv"], s["k_pe"]):
        t[:, dst] = t[:, src]


def _plain_fork(s):
    ps, rows, most = s["case"]["page"], *s["table"].shape
    table, n_pages, ref = s["table"], s["n_pages"], s["ref"]
    k = torch.arange(most, device=DEV)[None]
    ri = torch.arange(rows, device=DEV)
    # release
    keep = s["keep"]
    kept = torch.where(keep >= 0, torch.minimum((keep + ps - 1) // ps, n_pages), n_pages)
    gone = (k >= kept[:, None]) & (k < n_pages[:, None])
    ref -= torch.bincount(table[gone].long(), minlength=len(ref)).int()
    table[gone] = -1
    n_pages.copy_(kept)
    # fork
    src = s["source"].long()
    share = torch.where(src >= 0, (s["length"] + ps - 1) // ps, 0)
    new = k < share[:, None]
    table.copy_(torch.where(new, table[src.clamp(min=0)], table))
    ref += torch.bincount(table[new].long(), minlength=len(ref)).int()
    n_pages.copy_(torch.where(src >= 0, share, n_pages))
    # reserve: pages that overlap [length, new_length) have to be the row's own
    first, need = (s["length"] // ps)[:, None], ((s["new_length"] + ps - 1) // ps)[:, None]
    held = k < n_pages[:, None]
    pages = table.long().clamp(min=0)
    writes = held & (k >= first) & (k < need) & (ref[pages] > 1)
    writers = torch.bincount(table[writes].long(), minlength=len(ref))
    lowest = torch.full((len(ref),), rows, dtype=torch.long, device=DEV)
    lowest.scatter_reduce_(0, table[writes].long(),
                           ri[:, None].expand(rows, most)[writes], "amin")
    stays = (writers == ref)[pages] & (lowest[pages] == ri[:, None])
    swap = writes & ~stays
    take = swap | (~held & (k < need))
    order = torch.cumsum(take.flatten().long(), 0).view(rows, most) - 1
    free = torch.nonzero(ref == 0).flatten()
    fresh = free[order.clamp(min=0, max=len(free) - 1)]
    part = s["length"] % ps
    cut = swap & (k == first) & (part[:, None] > 0)
    copies = torch.full((rows, 3), -1, dtype=torch.int32, device=DEV)
    copies[:, 2] = 0
    some = cut.any(-1)
    at = first.clamp(max=most - 1).long()
    found = torch.cat([table.gather(1, at), fresh.gather(1, at).int(), part[:, None]], 1)
    copies = torch.where(some[:, None], found, copies)
    ref -= torch.bincount(table[swap].long(), minlength=len(ref)).int()
    ref[fresh[take]] = 1
    table.copy_(torch.where(take, fresh.int(), table))
    n_pages.copy_(torch.maximum(n_pages, need[:, 0]))
    _plain_copy(s, copies)
    s["copies"].copy_(copies)
    return table, n_pages, ref, s["copies"], s["c_kv"], s["k_pe"]


def _plain_compact(s):
    s["table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    table, ref = s["table"], s["ref"]
    used = ref > 0
    total = int(used.sum())
    p = torch.arange(len(ref), device=DEV)
    src = p[used & (p >= total)]
    dst = p[~used & (p < total)]
    to = p.clone()
    to[src] = dst
    held = torch.arange(table.shape[1], device=DEV)[None] < s["n_pages"][:, None]
    table.copy_(torch.where(held, to[table.long().clamp(min=0)].int(), table))
    ref[dst] = ref[src]
    ref[src] = 0
    rows = torch.full_like(src, s["case"]["page"])
    _plain_copy(s, torch.stack([src, dst, rows], 1))
    s["n_moves"].fill_(len(src))
    return table, s["n_pages"], ref, s["n_moves"], s["c_kv"], s["k_pe"]


def _key_rows(s, b):
    j = torch.arange(s["keys"][b], device=DEV)
    if s["table"] is None:
        return b * s["stride"] + j
    return s["table"][b, j // s["page"]].long() * s["page"] + j % s["page"]


def _plain_prefill(s):
    H, out, at = s["case"]["H"], s["out"], 0
    w = s["w_kv"].float()
    for b, n in enumerate(s["lens"]):
        rows = _key_rows(s, b)
        c, kp = s["c_kv"][rows].float(), s["k_pe"][rows].float()
        i = torch.arange(n, device=DEV)[:, None] + s["pre"][b]
        hidden = torch.arange(s["keys"][b], device=DEV)[None] > i
        for h0 in range(0, H, 8):
            hs = slice(h0, min(H, h0 + 8))
            kv = torch.matmul(c, w[hs].transpose(1, 2))            # [h, key, 256]
            q = s["q_nope"][at:at + n, hs].float().transpose(0, 1)
            qp = s["q_pe"][at:at + n, hs].float().transpose(0, 1)
            x = torch.matmul(q, kv[..., :128].transpose(1, 2)) + torch.matmul(qp, kp.T)
            x = (x * s["scale"]).masked_fill_(hidden, float("-inf"))
            x = torch.exp(x - x.max(-1, keepdim=True).values)
            x = x / x.sum(-1, keepdim=True)
            out[at:at + n, hs] = torch.matmul(x, kv[..., 128:]).transpose(0, 1).to(out.dtype)
        at += n
    return out


# --------------------------------------------------------------------------------------
# work and exact results
# --------------------------------------------------------------------------------------
def _pages_written(case):
    """(pages copied in part, rows copied) of a fork pass."""
    rows = [(x % case["page"]) * case["children"] for x in _lengths(case)]
    return sum(case["children"] for r in rows if r), sum(rows)


def work(case):
    op = case["op"]
    if op == "sample":
        es = 2 if case["dt"] == "bf16" else 4
        # the rows of the root and of the accepted nodes; a tree of these inputs accepts one
        # node or more, and a rejection reads the drafter's row
        rows = case["B"] * (1 if case["Q"] == 1 else 2)
        draft = case["B"] * case["V"] * 4 if case["draft"] != "none" and case["Q"] > 1 else 0
        return {"bytes": rows * case["V"] * es + draft + 5 * 4 * case["B"] * case["Q"],
                "flops": 4 * rows * case["V"]}
    es = 2 if case.get("dt", "bf16") == "bf16" else 4
    if op == "fork":
        row = (case["DL"] + case["DR"]) * es * case["layers"]
        n = case["parents"] * (1 + case["children"])
        share = sum(-(-x // case["page"]) for x in _lengths(case)) * case["children"]
        return {"bytes": 2 * row * _pages_written(case)[1] + 4 * (2 * share + 8 * n),
                "flops": 0}
    if op == "compact":
        # on average a page in use sits above the first `used` pages with the share free
        moved = case["used"] * (1 - case["used"] / case["pages"])
        page = (case["DL"] + case["DR"]) * es * case["layers"] * case["page"]
        return {"bytes": int(2 * moved * page) + 8 * case["pages"], "flops": 0}
    lens, pre = _ints(case["lens"]), _ints(case["prefixes"])
    H = case["H"]
    keys = sum(lens) + sum(pre)
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(lens, pre))
    return {"bytes": 2 * (keys * 576 + sum(lens) * H * (192 + 128) + H * 256 * 512),
            "flops": 2 * keys * 512 * H * 256 + 2 * pairs * H * (192 + 128)}


def exact(case, seed):
    op = case["op"]
    if op == "sample":
        return _exact_sample(case, seed)
    if op == "fork":
        return _exact_fork(case, seed)
    if op == "compact":
        return _exact_compact(case, seed)
    return _exact_prefill(case, seed)


def _exact_sample(case, seed):
    s = _sample_inputs(case, seed)
    B, Q, V = s["logits"].shape
    parent, tokens = s["parent"].cpu().numpy(), s["tokens"].cpu().numpy()
    u = s["uniforms"].cpu().numpy().astype(np.float64)
    temp = s["temp"].cpu().numpy().astype(np.float64)
    count = np.zeros(B, np.int32)
    path, emit = np.full((B, Q), -1, np.int32), np.full((B, Q), -1, np.int32)
    path[:, 0] = 0
    for b in range(B):
        node = 0
        while True:
            x = s["logits"][b, node].float().cpu().numpy().astype(np.float64)
            if temp[b] > 0:
                p = np.exp((x - x.max()) / temp[b])
                p /= p.sum()
            else:
                p = np.zeros(V)
                p[int(np.argmax(x))] = 1.0
            if s["probs"] is not None:
                row = node if s["by_node"] else int(count[b])
                q = (s["probs"][b, min(row, s["probs"].shape[1] - 1)].cpu().numpy()
                     .astype(np.float64))
                mass = 1.0
            step = -1
            for c in range(node + 1, Q):
                if parent[b, c] != node:
                    continue
                t = int(tokens[b, c])
                if s["probs"] is None:
                    if u[b, c] < p[t]:
                        step = c
                        break
                    p[t] = 0.0
                else:
                    if mass <= 0:
                        break
                    if u[b, c] * (q[t] / mass) < p[t]:
                        step = c
                        break
                    p = np.maximum(p - q / mass, 0.0)
                    mass -= q[t]
                    q[t] = p[t] = 0.0
                p /= p.sum()
            if step < 0:
                break
            emit[b, count[b]] = tokens[b, step]
            count[b] += 1
            path[b, count[b]] = step
            node = step
        total = np.cumsum(p)
        emit[b, count[b]] = min(V - 1, int(np.searchsorted(total, u[b, 0] * total[-1],
                                                           side="right")))
    return tuple(torch.from_numpy(a) for a in (count, path, emit))


def _exact_rows(case, num, seed, lists):
    """The cache after the copies (src page, dst page, rows)."""
    c, k = _cache(case, num, _gen(seed))
    ps = case["page"]
    for t in (c, k):
        pages = t.view(case["layers"], num, ps, t.shape[-1])
        for src, dst, n in lists:
            pages[:, dst, :n] = pages[:, src, :n]
    return c, k


def _exact_fork(case, seed):
    h = _fork_inputs(case, seed)
    ps = case["page"]
    table, ref, n_pages = h["table"].copy(), h["ref"].copy(), h["n_pages"].copy()
    rows = len(n_pages)
    for r in range(rows):
        if h["source"][r] >= 0:
            n = -(-int(h["length"][r]) // ps)
            table[r, :n] = table[h["source"][r], :n]
            ref[table[r, :n]] += 1
            n_pages[r] = n
    free = iter(np.flatnonzero(ref == 0).tolist())
    want = {}                                # shared page -> rows that write it
    for r in range(rows):
        for k in range(int(h["length"][r]) // ps, int(n_pages[r])):
            if ref[table[r, k]] > 1:
                want.setdefault(int(table[r, k]), []).append(r)
    keeper = {p: rs[0] for p, rs in want.items() if len(rs) == ref[p]}
    copies = np.full((rows, 3), -1, np.int32)
    copies[:, 2] = 0
    before = ref.copy()
    for r in range(rows):
        n, total = int(h["length"][r]), -(-int(h["new_length"][r]) // ps)
        for k in range(n // ps, total):
            old = int(table[r, k]) if k < n_pages[r] else -1
            if old >= 0 and (before[old] <= 1 or keeper.get(old) == r):
                continue
            new = next(free)
            if old >= 0:
                ref[old] -= 1
                if k == n // ps and n % ps:
                    copies[r] = (old, new, n % ps)
            ref[new] = 1
            table[r, k] = new
        n_pages[r] = max(int(n_pages[r]), total)
    c, k = _exact_rows(case, h["num"], seed, [x for x in copies.tolist() if x[0] >= 0])
    return (*(torch.from_numpy(a) for a in (table, n_pages, ref, copies)), c, k)


def _exact_compact(case, seed):
    h = _compact_inputs(case, seed)
    table, ref = h["table"], h["ref"]
    total = int((ref > 0).sum())
    src = [p for p in range(total, case["pages"]) if ref[p] > 0]
    dst = [p for p in range(total) if ref[p] == 0]
    to = dict(zip(src, dst))
    for r in range(len(table)):
        for i in range(int(h["n_pages"][r])):
            table[r, i] = to.get(int(table[r, i]), table[r, i])
    for a, b in to.items():
        ref[b], ref[a] = ref[a], 0
    c, k = _exact_rows(case, h["num"], seed, [(a, b, case["page"]) for a, b in to.items()])
    return (torch.from_numpy(table), torch.from_numpy(h["n_pages"]), torch.from_numpy(ref),
            torch.tensor([len(src)], dtype=torch.int32), c, k)


def _exact_prefill(case, seed):
    # the absorbed form: queries taken into the latent space, one head at a time
    s = _prefill_inputs(case, seed)
    out = torch.zeros((sum(s["lens"]), case["H"], 128), dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lens"]):
        at = int(s["q_start"][b])
        rows = _key_rows(s, b)
        c, kp = s["c_kv"][rows].double(), s["k_pe"][rows].double()
        last = s["pre"][b] + torch.arange(n, device=DEV)
        for h in range(case["H"]):
            w = s["w_kv"][h].double()
            ql = s["q_nope"][at:at + n, h].double() @ w[:128]
            x = (ql @ c.T + s["q_pe"][at:at + n, h].double() @ kp.T) * s["scale"]
            x[torch.arange(len(rows), device=DEV)[None] > last[:, None]] = float("-inf")
            out[at:at + n, h] = (torch.softmax(x, -1) @ c) @ w[128:].T
    return out
