"""Measured calls of the operators of a decode cycle over the latent cache.

Four operators, each in its plain form (elementary torch operations) and as a user's
program calls it in this package:

  shared  attention of sequences that share a long prefix, computed once for all of them
  rope    rotary positions: interleaved and half layouts, part of a head, scaled
  normed  norms of queries and keys with the position rotation, keys into the cache
  token   next tokens with temperature, top-k, top-p and min-p from given random numbers

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
        # Four samples of one short prompt on a small model: latency of one call.
        dict(name="shared_one", op="shared", H=16, Q=1, members="4", shared="700", own=40),
        # 64 samples of one long prompt, 16 heads, single tokens.
        dict(name="shared_samples", op="shared", H=16, Q=1, members="64", shared="8192",
             own=300),
        # A batch over three system prompts, one of them with a single user; 64 heads.
        dict(name="shared_prompts", op="shared", H=64, Q=1, members="24,1,39",
             shared="4000,5111,8150", own=1000),
        # Draft trees of nine nodes verified for samples of one prompt.
        dict(name="shared_trees", op="shared", H=16, Q=9, members="16,5",
             shared="8150,1777", own=500),
        # The query rope parts of a decode batch, interleaved pairs, contexts stretched by 32.
        dict(name="rope_decode", op="rope", T=64, H=64, d=64, at=0, rot=64, layout="pairs",
             scaling="yarn", factor=32.0, dt="bf16", far=100000),
        # A 4096-token prompt, 64 heads, the last 64 of 192 elements rotated.
        dict(name="rope_prompt", op="rope", T=4096, H=64, d=192, at=128, rot=64,
             layout="half", scaling="none", factor=1.0, dt="bf16", far=0),
        # An odd float32 layout: 5 heads of 80, the first 50 elements rotated.
        dict(name="rope_odd", op="rope", T=1001, H=5, d=80, at=0, rot=50, layout="pairs",
             scaling="linear", factor=4.0, dt="fp32", far=8000),
        # One new token for each of 64 sequences: queries and cache rows.
        dict(name="normed_decode", op="normed", H=64, DN=128, DR=64, DL=512,
             lens="1," * 63 + "1", prefixes="4096,100,777," * 21 + "5111", layout="pairs",
             dt="bf16"),
        # A ragged prompt batch, queries and cache rows.
        dict(name="normed_prompts", op="normed", H=64, DN=128, DR=64, DL=512,
             lens="1,700,33,1500,257,128", prefixes="900,0,1777,512,64,3000",
             layout="half", dt="bf16"),
        # One user, a 32000-token vocabulary: latency.
        dict(name="token_one", op="token", B=1, V=32000, dt="bf16", temp=0.8, k=50, p=0.9,
             m=0.0, spread=3.0),
        # Mixed requests over 163840 float32 logits: some greedy, top-k, top-p and min-p rows.
        dict(name="token_b64", op="token", B=64, V=163840, dt="fp32", temp=1.0, k=40, p=0.95,
             m=0.05, spread=3.0),
        # A full batch, nucleus sampling from flat distributions: the kept set is large.
        dict(name="token_b256", op="token", B=256, V=50257, dt="bf16", temp=1.0, k=0, p=0.95,
             m=0.0, spread=1.5),
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["shared", "shared", "rope", "normed", "token", "token"])
    if op == "shared":
        H = rng.choice([1, 5, 16, 64, 128])
        Q = rng.choice([1, 1, rng.randint(2, 16)])
        left = max(1, 6144 // (H * Q))
        members, shared = [], []
        for _ in range(rng.randint(1, 4)):
            n = min(left, _logint(rng, 1, 40))
            if n < 1:
                break
            left -= n
            members.append(n)
            shared.append(rng.choice([0, _logint(rng, 1, 8000), _logint(rng, 500, 8000)]))
        return dict(op=op, H=H, Q=Q, members=_text(members), shared=_text(shared),
                    own=_logint(rng, 1, 1200))
    if op == "rope":
        d = rng.choice([32, 64, 80, 128, 192, 256])
        rot = 2 * rng.randint(1, d // 2)
        at = rng.randint(0, d - rot)
        return dict(op=op, T=_logint(rng, 1, 2500), H=rng.choice([1, 5, 8, 64]), d=d, at=at,
                    rot=rot, layout=rng.choice(["half", "pairs"]),
                    scaling=rng.choice(["none", "linear", "ntk", "yarn", "wavelength"]),
                    factor=round(rng.uniform(1.0, 40.0), 2),
                    dt=rng.choice(["bf16", "fp32"]), far=rng.choice([0, 8000, 900000]))
    if op == "normed":
        B = rng.randint(1, 8)
        return dict(op=op, H=rng.choice([1, 5, 16, 64]), DN=rng.choice([0, 32, 128]),
                    DR=rng.choice([16, 64]), DL=rng.choice([64, 512]),
                    lens=_text(_logint(rng, 1, 400) for _ in range(B)),
                    prefixes=_text(rng.choice([0, _logint(rng, 1, 3000)]) for _ in range(B)),
                    layout=rng.choice(["half", "pairs"]), dt=rng.choice(["bf16", "fp32"]))
    B, V = _logint(rng, 1, 64), _logint(rng, 100, 163840)
    return dict(op=op, B=B, V=V, dt=rng.choice(["bf16", "fp32"]),
                temp=round(rng.uniform(0.4, 1.4), 2),
                k=rng.choice([0, 1, _logint(rng, 2, 2000)]),
                p=rng.choice([1.0, round(rng.uniform(0.1, 0.99), 3)]),
                m=rng.choice([0.0, round(rng.uniform(0.001, 0.3), 4)]),
                spread=round(rng.uniform(1.0, 4.0), 1))


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7907 + 29)
    return g


def _torch_dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _shared_inputs(case, seed):
    """Sequences of each group as a page pool leaves them: whole pages of the shared prefix
    named by all, the last, partly filled one copied for each, own pages behind."""
    H, Q, page = case["H"], case["Q"], 64
    members, shared = _ints(case["members"]), _ints(case["shared"])
    B = sum(members)
    r = np.random.default_rng([int(seed), 11])
    g = _gen(seed)
    group = np.repeat(np.arange(len(members)), members)
    start = np.concatenate([[0], np.cumsum(members)]).astype(np.int32)
    own_keys = r.integers(0, case["own"] + 1, B)
    prefix = np.array([shared[group[b]] for b in range(B)]) + own_keys
    need = -(-(prefix + Q) // page)
    whole = [s // page for s in shared]
    num = sum(whole) + int(sum(need[b] - whole[group[b]] for b in range(B))) + 3
    perm = r.permutation(num)
    table = np.zeros((B, int(need.max())), np.int32)
    at = 0
    for i, w in enumerate(whole):
        table[start[i]:start[i + 1], :w] = perm[at:at + w]
        at += w
    for b in range(B):
        n = int(need[b]) - whole[group[b]]
        table[b, whole[group[b]]:need[b]] = perm[at:at + n]
        at += n

    def randn(*shape, scale=1.0):
        x = torch.randn(shape, generator=g, device=DEV)
        return (x * scale).to(torch.bfloat16)

    c_kv, k_pe = randn(num * page, 512), randn(num * page, 64)
    for i, w in enumerate(whole):               # the copies of the partly filled page
        n = shared[i] % page
        src = int(table[start[i], w]) * page if n else 0
        for b in range(start[i] + 1, start[i + 1]):
            if n:
                dst = int(table[b, w]) * page
                c_kv[dst:dst + n] = c_kv[src:src + n]
                k_pe[dst:dst + n] = k_pe[src:src + n]
    # draft trees: node i hangs below one of the nodes just before it
    vis = np.zeros((B, Q, Q), bool)
    for b in range(B):
        for i in range(Q):
            if i:
                vis[b, i] = vis[b, r.integers(max(0, i - 4), i)]
            vis[b, i, i] = True
    bits = (vis.astype(np.uint64) << np.arange(Q, dtype=np.uint64)).sum(-1).astype(np.uint64)
    return dict(q_latent=randn(B, Q, H, 512, scale=0.25), q_pe=randn(B, Q, H, 64),
                c_kv=c_kv, k_pe=k_pe, table=_dev(table), vis=_dev(vis),
                anc=_dev(bits.view(np.int64)), prefix_len=_dev(prefix.astype(np.int32)),
                group_start=_dev(start), shared_len=_dev(np.array(shared, np.int32)),
                lens=prefix.tolist(), scale=192 ** -0.5)


def _rope_inputs(case, seed):
    g = _gen(seed)
    T, dt = case["T"], _torch_dt(case["dt"])
    r = np.random.default_rng([int(seed), 12])
    pos = np.arange(T) + (int(r.integers(0, case["far"] + 1)) if case["far"] else 0)
    if T <= 64:                                   # a decode batch: every token its own place
        pos = r.integers(0, case["far"] + 1, T)
    x = torch.randn((T, case["H"], case["d"]), generator=g, device=DEV).to(dt)
    return dict(x=x, positions=_dev(pos.astype(np.int32)))


def _normed_inputs(case, seed):
    g = _gen(seed)
    dt, page = _torch_dt(case["dt"]), 64
    lens, pre = _ints(case["lens"]), _ints(case["prefixes"])
    T, B = sum(lens), len(lens)
    need = [-(-(n + p) // page) for n, p in zip(lens, pre)]
    r = np.random.default_rng([int(seed), 13])
    first = [p // page for p in pre]              # pages before these are not touched
    num = sum(n - f for n, f in zip(need, first)) + 2
    perm = r.permutation(num)
    table = np.zeros((B, max(need)), np.int32)
    at = 0
    for b in range(B):
        n = need[b] - first[b]
        table[b, first[b]:need[b]] = perm[at:at + n]
        at += n

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV).to(dt)

    H, DN, DR, DL = case["H"], case["DN"], case["DR"], case["DL"]
    start = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    seq = np.repeat(np.arange(B), lens)
    key = np.concatenate([np.arange(p, p + n) for n, p in zip(lens, pre)])
    return dict(q=randn(T, H, DN + DR), kv=randn(T, DL + DR),
                q_weight=(1 + 0.3 * randn(DN + DR)).to(dt),
                kv_weight=(1 + 0.3 * randn(DL)).to(dt),
                c_kv=randn(num * page, DL), k_pe=randn(num * page, DR),
                q_start=_dev(start), prefix_len=_dev(np.array(pre, np.int32)),
                table=_dev(table), seq=_dev(seq), key=_dev(key))


def _token_inputs(case, seed):
    g = _gen(seed)
    B, V = case["B"], case["V"]
    logits = torch.randn((B, V), generator=g, device=DEV) * case["spread"]
    # a few likely tokens above the rest, as a trained model has them
    top = torch.randint(0, V, (B, 8), generator=g, device=DEV)
    rise = torch.rand((B, 8), generator=g, device=DEV) * (2 * case["spread"])
    logits.scatter_add_(1, top, rise)
    i = torch.arange(B, device=DEV)
    temp = torch.full((B,), case["temp"], device=DEV)
    k = torch.full((B,), case["k"], dtype=torch.int32, device=DEV)
    p = torch.full((B,), case["p"], device=DEV)
    m = torch.full((B,), case["m"], device=DEV)
    if case["k"] and case["p"] < 1 and case["m"] > 0:      # a mixed batch
        temp = torch.where(i % 8 == 7, torch.zeros_like(temp), temp)
        k = torch.where(i % 4 == 0, k, torch.zeros_like(k))
        p = torch.where(i % 4 <= 1, p, torch.ones_like(p))
        m = torch.where(i % 4 == 2, m, torch.zeros_like(m))
    return dict(logits=logits.to(_torch_dt(case["dt"])), temp=temp, k=k, p=p, m=m,
                uniforms=torch.rand((B,), generator=g, device=DEV))


_BASE, _CONTEXT = 10000.0, 4096


def prepare(case, seed):
    op = case["op"]
    if op == "shared":
        s = _shared_inputs(case, seed)
        B, Q, H = s["q_pe"].shape[:3]
        s["out"] = torch.zeros((B, Q, H, 512), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((B, Q, H), dtype=torch.float32, device=DEV)
    elif op == "rope":
        s = _rope_inputs(case, seed)
        s["out"] = torch.zeros_like(s["x"])
    elif op == "normed":
        s = _normed_inputs(case, seed)
        T, H, DN = s["q"].shape[0], case["H"], case["DN"]
        s["q_nope"] = torch.zeros((T, H, DN), dtype=s["q"].dtype, device=DEV)
        s["q_pe"] = torch.zeros((T, H, case["DR"]), dtype=s["q"].dtype, device=DEV)
    else:
        s = _token_inputs(case, seed)
        s["tokens"] = torch.zeros(case["B"], dtype=torch.int32, device=DEV)
        s["kept"] = torch.zeros(case["B"], dtype=torch.int32, device=DEV)
    s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    s["case"] = case
    return s


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if op == "shared":
        return _own_shared(s) if own else _plain_shared(s)
    if op == "rope":
        return _own_rope(s) if own else _plain_rope(s)
    if op == "normed":
        return _own_normed(s) if own else _plain_normed(s)
    return _own_token(s) if own else _plain_token(s)


def _own_shared(s):
    tv = _tv()
    tv.shared_attn(s["q_latent"], s["q_pe"], s["c_kv"], s["k_pe"], s["prefix_len"],
                   s["group_start"], s["shared_len"], s["out"], s["lse"], s["scale"],
                   max_prefix_len=max(s["lens"]), anc=s["anc"], page_table=s["table"],
                   status=s["status"])
    return s["out"], s["lse"]


def _own_scaling(case):
    tv = _tv()
    if case["op"] == "normed" or case["scaling"] == "none":
        return tv.rope_scaling(base=_BASE)
    kind = {"linear": tv.ROPE_LINEAR, "ntk": tv.ROPE_NTK, "yarn": tv.ROPE_YARN,
            "wavelength": tv.ROPE_WAVELENGTH}[case["scaling"]]
    return tv.rope_scaling(base=_BASE, kind=kind, factor=case["factor"],
                           original_context=_CONTEXT)


def _own_layout(case):
    tv = _tv()
    return tv.ROPE_HALF if case["layout"] == "half" else tv.ROPE_INTERLEAVED


def _own_rope(s):
    c = s["case"]
    _tv().rope(s["x"], s["out"], s["positions"], layout=_own_layout(c), rot_offset=c["at"],
               rot_dim=c["rot"], scaling=_own_scaling(c))
    return s["out"]


def _own_normed(s):
    c = s["case"]
    _tv().norm_rope(s["q"], s["kv"], s["q_start"], s["prefix_len"], s["q_nope"], s["q_pe"],
                    s["c_kv"], s["k_pe"], q_weight=s["q_weight"], kv_weight=s["kv_weight"],
                    layout=_own_layout(c), scaling=_own_scaling(c), page_table=s["table"],
                    status=s["status"])
    return s["q_nope"], s["q_pe"], s["c_kv"], s["k_pe"]


def _own_token(s):
    _tv().token_sample(s["logits"], s["uniforms"], s["tokens"], temperature=s["temp"],
                       top_k=s["k"], top_p=s["p"], min_p=s["m"], kept=s["kept"],
                       status=s["status"])
    return s["tokens"], s["kept"]


def _plain_shared(s):
    B, Q, H = s["q_pe"].shape[:3]
    for b in range(B):
        n = s["lens"][b] + Q
        j = torch.arange(n, device=DEV)
        rows = s["table"][b, j // 64].long() * 64 + j % 64
        c, kp = s["c_kv"][rows].float(), s["k_pe"][rows].float()
        x = torch.matmul(s["q_latent"][b].float(), c.T)           # [Q, H, key]
        x = (x + torch.matmul(s["q_pe"][b].float(), kp.T)) * s["scale"]
        x[:, :, n - Q:].masked_fill_(~s["vis"][b][:, None], float("-inf"))
        top = x.max(-1, keepdim=True).values
        e = torch.exp(x - top)
        z = e.sum(-1, keepdim=True)
        s["out"][b] = (torch.matmul(e, c) / z).to(s["out"].dtype)
        s["lse"][b] = (top + torch.log(z))[..., 0]
    return s["out"], s["lse"]


def _frequencies(case):
    """Angle per position of each pair, and the factor on cos and sin."""
    d = case["rot"] if case["op"] == "rope" else case["DR"]
    k = torch.arange(d // 2, dtype=torch.float64, device=DEV)
    inv = _BASE ** (-2.0 * k / d)
    kind = case.get("scaling", "none")
    f = case.get("factor", 1.0)
    if kind == "linear":
        return inv / f, 1.0
    if kind == "ntk":
        return (_BASE * f ** (d / max(1, d - 2))) ** (-2.0 * k / d), 1.0
    if kind == "yarn":
        # pairs that turn more than 32 times over the trained context keep their frequency,
        # those below one turn are stretched, a ramp over the pair's index between
        lo, hi = (d * math.log(_CONTEXT / (2 * math.pi * turns)) / (2 * math.log(_BASE))
                  for turns in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), d - 1)
        ramp = ((k - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return inv * (1 - ramp) + inv / f * ramp, 0.1 * math.log(f) + 1.0
    if kind == "wavelength":
        turns = _CONTEXT * inv / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return inv * keep + inv / f * (1 - keep), 1.0
    return inv, 1.0


def _turned(case, x, positions):
    """x [T, heads, d] in 32 bits, rotated; angles in 64."""
    inv, mag = _frequencies(case)
    a = positions.double()[:, None] * inv[None]
    cos, sin = (torch.cos(a) * mag).float()[:, None], (torch.sin(a) * mag).float()[:, None]
    n = x.shape[-1] // 2
    if case["layout"] == "half":
        x0, x1 = x[..., :n], x[..., n:]
        return torch.cat([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1)
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack([x0 * cos - x1 * sin, x1 * cos + x0 * sin], -1).flatten(-2)


def _plain_rope(s):
    c, out = s["case"], s["out"]
    part = slice(c["at"], c["at"] + c["rot"])
    out.copy_(s["x"])
    out[..., part] = _turned(c, s["x"][..., part].float(), s["positions"]).to(out.dtype)
    return out


def _normalised(x, w):
    y = x.float()
    return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w.float()


def _plain_normed(s):
    c = s["case"]
    DN, DL = c["DN"], c["DL"]
    dt = s["q"].dtype
    q = _normalised(s["q"], s["q_weight"])
    s["q_nope"].copy_(q[..., :DN].to(dt))
    s["q_pe"].copy_(_turned(c, q[..., DN:], s["key"]).to(dt))
    rows = s["table"][s["seq"], s["key"] // 64].long() * 64 + s["key"] % 64
    s["c_kv"][rows] = _normalised(s["kv"][:, :DL], s["kv_weight"]).to(dt)
    kp = s["kv"][:, DL:].float()[:, None]
    s["k_pe"][rows] = _turned(c, kp, s["key"])[:, 0].to(dt)
    return s["q_nope"], s["q_pe"], s["c_kv"], s["k_pe"]


def _plain_token(s):
    # 64 bits: the cut of a nucleus and the drawn token turn on running sums
    x = s["logits"].double()
    B, V = x.shape
    t = s["temp"].double()[:, None]
    y = x / torch.where(t > 0, t, torch.ones_like(t))
    w = torch.exp(y - y.max(-1, keepdim=True).values)
    ranked, order = torch.sort(x, dim=-1, descending=True, stable=True)
    ws = w.gather(1, order)
    at = torch.arange(V, device=DEV)[None]
    k = s["k"][:, None]
    keep = (k <= 0) | (at < k)
    ws = torch.where(keep, ws, torch.zeros_like(ws))
    before = torch.cumsum(ws, -1) - ws
    p = s["p"].double()[:, None]
    keep &= (p >= 1) | (before < p * ws.sum(-1, keepdim=True)) | (at == 0)
    m = s["m"].double()[:, None]
    keep &= (m <= 0) | (ws >= m) | (at == 0)
    keep = torch.where(t > 0, keep, at == 0)
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    w = torch.where(kept, w, torch.zeros_like(w))
    run_sum = torch.cumsum(w, -1)
    aim = s["uniforms"].double()[:, None] * run_sum[:, -1:]
    drawn = (run_sum <= aim).sum(-1).clamp(max=V - 1)
    s["tokens"].copy_(drawn.int())
    s["kept"].copy_(keep.sum(-1).int())
    return s["tokens"], s["kept"]


# --------------------------------------------------------------------------------------
# work and exact results
# --------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "shared":
        # the shared keys once for each group, every sequence's own keys (half of `own` on
        # average) and tree once; scores and sums for every visible pair
        H, Q = case["H"], case["Q"]
        members, shared = _ints(case["members"]), _ints(case["shared"])
        B = sum(members)
        keys = sum(shared) + B * (case["own"] // 2 + Q)
        pairs = Q * (sum(n * x for n, x in zip(members, shared)) + B * (case["own"] // 2 + 1))
        return {"bytes": 2 * 576 * keys + B * Q * H * (2 * 576 + 2 * 512 + 4),
                "flops": 2 * H * pairs * (576 + 512)}
    es = 2 if case["dt"] == "bf16" else 4
    if op == "rope":
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * case["d"] * es + 4 * case["T"], "flops": 3 * n * case["rot"]}
    if op == "normed":
        T = sum(_ints(case["lens"]))
        row = case["H"] * (case["DN"] + case["DR"]) + case["DL"] + case["DR"]
        return {"bytes": 2 * T * row * es, "flops": 7 * T * row}
    return {"bytes": case["B"] * case["V"] * es, "flops": 4 * case["B"] * case["V"]}


def exact(case, seed):
    op = case["op"]
    if op == "shared":
        return _exact_shared(case, seed)
    if op == "rope":
        return _exact_rope(case, seed)
    if op == "normed":
        return _exact_normed(case, seed)
    return _exact_token(case, seed)


def _exact_shared(case, seed):
    # shared keys and own keys apart, joined by their sums
    s = _shared_inputs(case, seed)
    B, Q, H = s["q_pe"].shape[:3]
    start, shared = s["group_start"].tolist(), s["shared_len"].tolist()
    cache = torch.cat([s["c_kv"], s["k_pe"]], -1)
    q = torch.cat([s["q_latent"], s["q_pe"]], -1).double() * s["scale"]
    out = torch.zeros((B, Q, H, 512), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Q, H), dtype=torch.float64, device=DEV)
    pages = cache.view(-1, 64, 576)
    for i, n in enumerate(shared):
        first = start[i]
        common = pages[s["table"][first, :-(-n // 64)].long()].reshape(-1, 576)[:n].double()
        for b in range(first, start[i + 1]):
            total = s["lens"][b] + Q
            mine = pages[s["table"][b, :-(-total // 64)].long()].reshape(-1, 576)[n:total]
            mine = mine.double()
            a = q[b].reshape(Q * H, 576)
            y = a @ mine.T
            y = y.view(Q, H, -1)
            y[:, :, total - Q - n:] += torch.where(s["vis"][b], 0.0, -math.inf)[:, None]
            both = torch.cat([(a @ common.T).view(Q, H, -1), y], -1)
            lse[b] = torch.logsumexp(both, -1)
            prob = torch.exp(both - lse[b][..., None])
            out[b] = prob[..., :n] @ common[:, :512] + prob[..., n:] @ mine[:, :512]
    return out, lse


def _exact_angles(case, positions):
    d = case["rot"] if case["op"] == "rope" else case["DR"]
    kind, f = case.get("scaling", "none"), case.get("factor", 1.0)
    rates, mag = [], 1.0
    for k in range(d // 2):
        rate = math.exp(-2.0 * k / d * math.log(_BASE))
        if kind == "linear":
            rate /= f
        elif kind == "ntk":
            rate = math.exp(-2.0 * k / d * (math.log(_BASE) + d / max(1, d - 2) * math.log(f)))
        elif kind == "yarn":
            mag = 0.1 * math.log(f) + 1.0
            bound = [d * math.log(_CONTEXT / (2 * math.pi * n)) / (2 * math.log(_BASE))
                     for n in (32.0, 1.0)]
            lo, hi = max(0, math.floor(bound[0])), min(d - 1, math.ceil(bound[1]))
            share = min(1.0, max(0.0, (k - lo) / max(hi - lo, 1e-3)))
            rate = rate * (1 - share) + rate / f * share
        elif kind == "wavelength":
            turns = _CONTEXT * rate / (2 * math.pi)
            if turns < 1.0:
                rate /= f
            elif turns < 4.0:
                t = (turns - 1.0) / 3.0
                rate = (1 - t) * rate / f + t * rate
        rates.append(rate)
    a = torch.outer(positions.double().cpu(), torch.tensor(rates, dtype=torch.float64))
    return torch.polar(torch.full_like(a, mag), a).to(DEV)


def _exact_turn(case, x, positions):
    turn = _exact_angles(case, positions)[:, None]
    n = x.shape[-1] // 2
    if case["layout"] == "half":
        z = torch.complex(x[..., :n].contiguous(), x[..., n:].contiguous()) * turn
        return torch.cat([z.real, z.imag], -1)
    z = torch.view_as_complex(x.contiguous().view(*x.shape[:-1], n, 2)) * turn
    return torch.view_as_real(z).reshape(x.shape)


def _exact_rope(case, seed):
    s = _rope_inputs(case, seed)
    out = s["x"].double()
    part = out[..., case["at"]:case["at"] + case["rot"]]
    out[..., case["at"]:case["at"] + case["rot"]] = _exact_turn(case, part, s["positions"])
    return out


def _exact_normed(case, seed):
    s = _normed_inputs(case, seed)
    DN, DL = case["DN"], case["DL"]
    q = s["q"].double()
    q = q / torch.sqrt(torch.square(q).sum(-1, keepdim=True) / q.shape[-1] + 1e-6)
    q = q * s["q_weight"].double()
    c = s["kv"][:, :DL].double()
    c = c / torch.sqrt(torch.square(c).sum(-1, keepdim=True) / DL + 1e-6)
    c_kv, k_pe = s["c_kv"].double(), s["k_pe"].double()
    pages = s["table"].long()[s["seq"], torch.div(s["key"], 64, rounding_mode="floor")]
    at = pages * 64 + torch.remainder(s["key"], 64)
    c_kv.index_copy_(0, at, c * s["kv_weight"].double())
    turned = _exact_turn(case, s["kv"][:, None, DL:].double(), s["key"])
    k_pe.index_copy_(0, at, turned[:, 0])
    return q[..., :DN], _exact_turn(case, q[..., DN:], s["key"]), c_kv, k_pe


def _exact_token(case, seed):
    s = {n: t.cpu().numpy() if t.dtype != torch.bfloat16 else t.float().cpu().numpy()
         for n, t in _token_inputs(case, seed).items()}
    tokens, kept = [], []
    for b in range(case["B"]):
        x = s["logits"][b].astype(np.float64)
        if s["temp"][b] <= 0:
            tokens.append(int(np.argmax(x)))
            kept.append(1)
            continue
        w = np.exp((x - x.max()) / np.float64(s["temp"][b]))
        rank = np.argsort(-x, kind="stable")
        n = len(x)
        if s["k"][b] > 0:
            n = min(n, int(s["k"][b]))
        if s["p"][b] < 1:
            run_sum = np.cumsum(w[rank[:n]])
            # tokens up to the first whose running sum reaches the share
            n = 1 + int(np.searchsorted(run_sum[:-1], np.float64(s["p"][b]) * run_sum[-1]))
        if s["m"][b] > 0:
            n = max(1, min(n, int((w[rank[:n]] >= np.float64(s["m"][b])).sum())))
        chosen = np.sort(rank[:n])
        total = np.cumsum(w[chosen])
        i = int(np.searchsorted(total, np.float64(s["uniforms"][b]) * total[-1], side="right"))
        tokens.append(int(chosen[min(i, n - 1)]))
        kept.append(n)
    return (torch.tensor(tokens, dtype=torch.int32), torch.tensor(kept, dtype=torch.int32))
