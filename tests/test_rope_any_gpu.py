"""GPU tests of tv_rope and tv_norm_rope against their formulas in 64 bits.

Tolerance.  With |a| + |b| the size of an element's pair and M the magnitude: a float32 result is
within 2^-23 of itself (one unit) of the formula in double; bf16 within 2^-20 M (|a| + |b|) before
its rounding, 2^-8 of itself.  The formula's own angle pos * f_k carries two roundings of 2^-53
(and the model's f_k another few), which turn a pair by up to pos * 2^-50.  A normalised element
is a float32 product of four factors, one of them from a sum of n squares: within (n/32 + 16)
2^-24 of itself, and a pair of them likewise.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import decode_model as dm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
KIND = dict(plain=tv.ROPE_PLAIN, linear=tv.ROPE_LINEAR, ntk=tv.ROPE_NTK, yarn=tv.ROPE_YARN,
            wavelength=tv.ROPE_WAVELENGTH)
LAYOUT = dict(half=tv.ROPE_HALF, pairs=tv.ROPE_INTERLEAVED)


def rotated(x, positions, layout, mag, f, dt, more=0.0):
    """The rotated part x [T,H,rot] (float64) and how far a result of type dt may be off."""
    pos = np.asarray(positions, np.float64)
    y = dm.turn(x, pos[:, None] * f[None], layout, mag)
    size = dm.pair_size(x, layout) * mag
    unit = 2.0 ** -8 if dt is torch.bfloat16 else 2.0 ** -23
    slack = (2.0 ** -20 if dt is torch.bfloat16 else 0.0) + np.abs(pos)[:, None, None] * 2.0 ** -50
    return y, unit * np.abs(y) + (slack + more) * size + 1e-45


def turn(x, positions, out=None, **kw):
    d = x.cuda() if not x.is_cuda else x
    out = torch.full_like(d, -77.0) if out is None else out
    tv.rope(d, out, torch.tensor(np.asarray(positions), dtype=torch.int32).cuda(), **kw)
    torch.cuda.synchronize()
    return out


CASES = [  # T, H, d, at, rot, layout, kind, factor, first position
    (1, 1, 2, 0, 2, "pairs", "plain", 1.0, 7), (1, 1, 2, 0, 2, "half", "plain", 1.0, 0),
    (5, 3, 64, 0, 64, "half", "plain", 1.0, 0), (7, 64, 64, 0, 64, "pairs", "yarn", 32.0, 5000),
    (33, 5, 80, 0, 50, "pairs", "linear", 4.0, 8000), (9, 4, 80, 30, 50, "half", "ntk", 8.0, 11),
    (300, 16, 192, 128, 64, "half", "plain", 1.0, 100000), (700, 2, 192, 128, 64, "pairs", "wavelength", 8.0, 3),
    (4, 7, 66, 1, 34, "half", "yarn", 2.5, 70), (3, 2, 512, 0, 512, "half", "plain", 1.0, 9),
    (3, 2, 512, 0, 512, "pairs", "ntk", 3.0, 9), (2, 3, 2000, 16, 480, "pairs", "plain", 1.0, 900000),
    (400, 1, 16, 8, 8, "pairs", "plain", 1.0, 2 ** 31 - 500), (310, 9, 24, 0, 16, "half", "yarn", 1.0, 0),
]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_rope(i, dt):
    T, H, d, at, rot, layout, kind, factor, first = CASES[i]
    x = torch.randn((T, H, d), generator=torch.Generator().manual_seed(i)).to(dt)
    pos = first + np.arange(T)
    sc = tv.rope_scaling(kind=KIND[kind], factor=factor)
    kw = dict(layout=LAYOUT[layout], rot_offset=at, rot_dim=rot, scaling=sc)
    out = turn(x, pos, **kw).cpu()
    f, mag = dm.frequencies(rot, kind=kind, factor=factor), dm.magnitude(kind, factor)
    part = slice(at, at + rot)
    ref, tol = rotated(x[..., part].double().numpy(), pos, layout, mag, f, dt)
    err = np.abs(out[..., part].double().numpy() - ref)
    assert (err <= tol).all(), float((err - tol).max())
    keep = torch.ones(d, dtype=torch.bool)
    keep[part] = False
    assert torch.equal(out[..., keep], x[..., keep])
    # in place, and back again
    y = x.cuda()
    turn(y, pos, out=y, **kw)
    assert torch.equal(y.cpu(), out)
    if kind == "plain":
        back = turn(out.cuda(), pos, inverse=True, **kw).cpu().double().numpy()[..., part]
        z, tol2 = rotated(out[..., part].double().numpy(), -pos.astype(np.float64), layout, mag, f, dt)
        assert (np.abs(back - z) <= tol2).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_half_layout_is_rope_neox(dt):
    B, Q, H, D = 3, 5, 6, 64
    x = torch.randn((B, Q, H, D), generator=torch.Generator().manual_seed(3)).to(dt).cuda()
    prefix = torch.tensor([0, 700, 123456], dtype=torch.int32, device="cuda")
    want = torch.empty_like(x)
    tv.rope_neox(x, want, prefix, None)
    pos = (prefix[:, None] + torch.arange(Q, device="cuda")[None]).flatten().int()
    out = torch.empty_like(x)
    tv.rope(x.view(-1, H, D), out.view(-1, H, D), pos)
    if dt is torch.float32:
        assert torch.equal(out, want)
    else:  # a rounding may fall the other way, one in some thousands
        assert (out != want).float().mean() < 1e-3
        assert ((out - want).abs() <= 2.0 ** -7 * want.abs() + 1e-30).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_strides_and_alignments(dt, layout):
    T, H, d = 20, 6, 64
    g = torch.Generator().manual_seed(4)
    wide = torch.randn((H, T, 200), generator=g).to(dt).cuda()
    pos = np.arange(T) * 31
    for at in (0, 8, 3, 33):                      # slices of one buffer, heads outermost
        x = wide[:, :, at:at + d].transpose(0, 1)
        buf = torch.full((T, H, 100), -77.0, dtype=dt, device="cuda")
        out = buf[:, :, at:at + d]
        turn(x, pos, out=out, layout=LAYOUT[layout])
        ref, tol = rotated(x.double().cpu().numpy(), pos, layout, 1.0, dm.frequencies(d), dt)
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
        rest = torch.cat([buf[:, :, :at], buf[:, :, at + d:]], -1)
        assert (rest == -77.0).all()
    y = wide[:, :, 5:5 + d].transpose(0, 1)       # in place within a buffer
    ref, tol = rotated(y.double().cpu().numpy(), pos, layout, 1.0, dm.frequencies(d), dt)
    turn(y, pos, out=y, layout=LAYOUT[layout])
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


def test_gradient_is_the_inverse_turn():
    # d(w . out)/dx is the inverse turn of w, against differences of the formula
    T, H, d = 4, 2, 12
    g = torch.Generator().manual_seed(6)
    x, w = (torch.randn((T, H, d), generator=g) for _ in range(2))
    pos = np.array([0, 3, 77, 5000])
    sc = tv.rope_scaling(kind=tv.ROPE_YARN, factor=4.0)
    f, mag = dm.frequencies(8, kind="yarn", factor=4.0), dm.magnitude("yarn", 4.0)

    def loss(v):
        y = v.copy()
        y[..., 2:10] = dm.turn(v[..., 2:10], pos[:, None] * f[None], "pairs", mag)
        return (y * w.double().numpy()).sum()
    grad = turn(w, pos, layout=tv.ROPE_INTERLEAVED, rot_offset=2, rot_dim=8, scaling=sc,
                inverse=True).cpu().double().numpy()
    base = x.double().numpy()
    for at in np.ndindex(T, H, d):                # (the loss is linear: any step is exact)
        e = np.zeros_like(base)
        e[at] = 1.0
        slope = loss(base + e) - loss(base)
        assert abs(slope - grad[at]) <= 2.0 ** -22 * 4 + 5000 * 2.0 ** -50 * 8


def test_negative_positions_and_many_tokens():
    x = torch.randn((3000, 1, 32), generator=torch.Generator().manual_seed(7)).bfloat16()
    pos = np.arange(3000) - 1500
    out = turn(x, pos).double().cpu().numpy()
    ref, tol = rotated(x.double().numpy(), pos, "half", 1.0, dm.frequencies(32), torch.bfloat16)
    assert (np.abs(out - ref) <= tol).all()


# ---- norms -----------------------------------------------------------------------------
def batch(seed, lens, prefixes, H, DN, DR, DL, dt, paged=True, tail=0, page=64, qw=True, kvw=True,
          kw=False, rot=None, layout="half", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    B, T = len(lens), sum(lens) + tail

    def randn(*shape):
        return (torch.randn(shape, generator=g) * scale).to(dt)
    keys = [n + p for n, p in zip(lens, prefixes)]
    need = [-(-k // page) for k in keys]
    table, stride, rows = None, 0, 0
    if paged:
        perm = r.permutation(sum(need) + 1)
        table = np.full((B, max(need) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        rows = len(perm) * page
    else:
        stride = max(keys) + 2
        rows = B * stride
    s = dict(lens=lens, prefixes=prefixes, H=H, DN=DN, DR=DR, DL=DL, dt=dt, table=table,
             stride=stride, page=page, rows=rows, rot=rot or DR, layout=layout,
             q=randn(T, H, DN + DR), kv=randn(T, DL + DR),
             q_weight=1 + 0.3 * randn(DN + DR) if qw else None,
             kv_weight=1 + 0.3 * randn(DL) if kvw else None,
             k_weight=1 + 0.3 * randn(DR) if kw else None)
    for n in ("q_weight", "kv_weight", "k_weight"):
        s[n] = None if s[n] is None else s[n].to(dt)
    s["start"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return s


def apply(s, status=0, queries=True, keys=True, depth=None, prefixes=None, **kw):
    def put(t):
        return None if t is None else (torch.from_numpy(t) if isinstance(t, np.ndarray)
                                       else t).cuda()
    T, H, dt = s["q"].shape[0], s["H"], s["dt"]
    o = dict(q_nope=torch.full((T, H, s["DN"]), -77.0, dtype=dt, device="cuda"),
             q_pe=torch.full((T, H, s["DR"]), -77.0, dtype=dt, device="cuda"),
             c_kv=torch.full((s["rows"], s["DL"]), -77.0, dtype=dt, device="cuda"),
             k_pe=torch.full((s["rows"], s["DR"]), -77.0, dtype=dt, device="cuda"))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pre = np.asarray(s["prefixes"] if prefixes is None else prefixes, np.int32)
    tv.norm_rope(put(s["q"]) if queries else None, put(s["kv"]) if keys else None,
                 put(s["start"]), put(pre), o["q_nope"] if s["DN"] else None, o["q_pe"],
                 o["c_kv"], o["k_pe"], q_weight=put(s["q_weight"]), kv_weight=put(s["kv_weight"]),
                 k_weight=put(s["k_weight"]), rot_dim=s["rot"], layout=LAYOUT[s["layout"]],
                 depth=put(depth), page_table=put(s["table"]), page_size=s["page"],
                 kv_stride_b=s["stride"], status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return {k: v.double().cpu().numpy() for k, v in o.items()}


def near(got, ref, tol, what):
    assert (np.abs(got - ref) <= tol).all(), (what, float((np.abs(got - ref) - tol).max()))


def compare(s, o, eps=1e-6, depth=None, skip=(), queries=True, keys=True):
    DN, DL, dt, rot = s["DN"], s["DL"], s["dt"], s["rot"]
    unit = 2.0 ** -8 if dt is torch.bfloat16 else 2.0 ** -23
    f = dm.frequencies(rot)
    left = np.ones(s["rows"], bool)
    done = np.zeros(s["q"].shape[0], bool)
    for b, (n, P) in enumerate(zip(s["lens"], s["prefixes"])):
        lo = int(s["start"][b])
        t = np.array([i for i in range(n) if lo + i not in skip], int)
        if not len(t):
            continue
        j = P + t
        pos = P + (t if depth is None else np.asarray(depth)[lo + t])
        done[lo + t] = True

        def part(x, w, what):                     # normalised values and their relative error
            x = x.double().numpy()
            more = 0.0 if w is None else (x.shape[-1] / 32 + 16) * 2.0 ** -24
            return dm.norm(x, None if w is None else w.double().numpy(), eps), more

        def turned(x, more, got, what):           # x [t, heads, DR]
            y, tol = rotated(x[..., :rot], pos, s["layout"], 1.0, f, dt, more)
            near(got[..., :rot], y, tol, what)
            near(got[..., rot:], x[..., rot:], (unit + more) * np.abs(x[..., rot:]), what)
        if queries:
            y, more = part(s["q"][lo + t], s["q_weight"], "q")
            if DN:
                near(o["q_nope"][lo + t], y[..., :DN], (unit + more) * np.abs(y[..., :DN]), "nope")
            turned(y[..., DN:], more, o["q_pe"][lo + t], "q_pe")
        if keys:
            row = (s["table"][b, j // s["page"]].astype(np.int64) * s["page"] + j % s["page"]
                   if s["table"] is not None else b * s["stride"] + j)
            left[row] = False
            y, more = part(s["kv"][lo + t, :DL], s["kv_weight"], "kv")
            near(o["c_kv"][row], y, (unit + more) * np.abs(y), "c_kv")
            y, more = part(s["kv"][lo + t, DL:], s["k_weight"], "k")
            turned(y[:, None], more, o["k_pe"][row][:, None], "k_pe")
    assert (o["c_kv"][left] == -77.0).all() and (o["k_pe"][left] == -77.0).all()
    if not queries:
        done[:] = False
    assert (o["q_pe"][~done] == -77.0).all() and (o["q_nope"][~done] == -77.0).all()


NORMED = [
    dict(lens=[1], prefixes=[0], H=1, DN=0, DR=2, DL=1),
    dict(lens=[1] * 9, prefixes=list(range(0, 900, 100)), H=16, DN=128, DR=64, DL=512),
    dict(lens=[5, 0, 70, 1], prefixes=[63, 9, 100, 64], H=5, DN=32, DR=16, DL=64, layout="pairs"),
    dict(lens=[400], prefixes=[0], H=64, DN=128, DR=64, DL=512, kw=True, layout="pairs"),
    dict(lens=[3, 4], prefixes=[10, 0], H=3, DN=7, DR=10, DL=33, rot=6, layout="pairs", kw=True),
    dict(lens=[3, 4], prefixes=[10, 0], H=3, DN=8, DR=48, DL=40, rot=32, page=16),
    dict(lens=[2, 30], prefixes=[500, 0], H=8, DN=64, DR=64, DL=1024, qw=False, paged=False),
    dict(lens=[20], prefixes=[1], H=2, DN=16, DR=64, DL=2048, kvw=False),
    dict(lens=[4, 1], prefixes=[7, 3], H=40, DN=512, DR=64, DL=512, tail=3),
]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(NORMED)))
def test_norm_rope(i, dt):
    s = batch(50 + i, dt=dt, **NORMED[i])
    compare(s, apply(s))


@pytest.mark.parametrize("queries,keys", [(True, False), (False, True)])
def test_one_side_alone(queries, keys):
    s = batch(70, [3, 9], [60, 2], 4, 32, 64, 128, torch.bfloat16)
    compare(s, apply(s, queries=queries, keys=keys), queries=queries, keys=keys)


def test_depths_of_a_draft_tree():
    s = batch(71, [9, 9], [200, 31], 8, 0, 64, 512, torch.bfloat16, qw=False)
    depth = np.array([0, 1, 1, 2, 2, 3, 1, 2, 4] * 2, np.int32)
    compare(s, apply(s, depth=depth), depth=depth)
    depth[9 + 4] = -1
    compare(s, apply(s, depth=depth), depth=depth, skip=[13])


def test_zeros_and_large_values():
    s = batch(72, [6], [0], 3, 16, 16, 64, torch.float32)
    s["q"][1], s["kv"][1] = 0.0, 0.0
    s["q"][2] *= 1e15
    s["kv"][3] *= 1e-12
    compare(s, apply(s, eps=1e-5), eps=1e-5)


def test_keys_outside_the_cache():
    s = batch(73, [4, 5], [62, 126], 2, 16, 16, 64, torch.bfloat16)
    s["table"][0, 1] = -1                 # keys 64 and 65 of sequence 0
    s["table"][1, 2] = 10 ** 6            # keys 128 .. of sequence 1
    o = apply(s, status=tv.TV_ERR_BOUNDS)
    hit = [s["table"][0, 0] * 64 + j for j in (62, 63)] + \
        [s["table"][1, 1] * 64 + j for j in (62, 63)]
    written = np.flatnonzero((o["c_kv"] != -77.0).any(-1))
    assert sorted(hit) == written.tolist()
    assert (o["q_pe"] != -77.0).all()     # the queries are there all the same


def test_a_negative_prefix_leaves_its_tokens():
    s = batch(74, [3, 2, 4], [5, 6, 7], 2, 16, 16, 64, torch.bfloat16)
    o = apply(s, status=tv.TV_ERR_BOUNDS, prefixes=[5, -1, 7])
    compare(s, o, skip=[3, 4])


def test_strided_inputs_share_a_buffer():
    # queries and keys as two parts of one projection's output
    H, DN, DR, DL, T = 4, 32, 16, 64, 10
    s = batch(75, [10], [3], H, DN, DR, DL, torch.bfloat16)
    both = torch.cat([s["q"].flatten(1), s["kv"]], -1).cuda()
    q = both[:, :H * (DN + DR)].view(T, H, DN + DR)
    kv = both[:, H * (DN + DR):]
    o = apply(s)
    out = {k: torch.full(v.shape, -77.0, dtype=torch.bfloat16, device="cuda")
           for k, v in o.items()}
    i32 = dict(dtype=torch.int32, device="cuda")
    tv.norm_rope(q, kv, torch.from_numpy(s["start"]).cuda(), torch.tensor([3], **i32),
                 out["q_nope"], out["q_pe"], out["c_kv"], out["k_pe"],
                 q_weight=s["q_weight"].cuda(), kv_weight=s["kv_weight"].cuda(),
                 page_table=torch.from_numpy(s["table"]).cuda())
    for k in o:
        assert np.array_equal(out[k].double().cpu().numpy(), o[k])


def test_cache_rows_within_wider_ones():
    # both arrays are parts of one row of 2 + 64 + 6 + 16 + 8 elements, at any alignment
    for dt in (torch.bfloat16, torch.float32):
        for off in (0, 8, 2, 3):
            s = batch(77, [5, 3], [60, 0], 3, 16, 16, 64, dt)
            want = apply(s)
            wide = torch.full((s["rows"], 128), -77.0, dtype=dt, device="cuda")
            c, k = wide[:, off:off + 64], wide[:, off + 72:off + 88]
            T, H = s["q"].shape[:2]
            i32 = dict(dtype=torch.int32, device="cuda")
            tv.norm_rope(None, s["kv"].cuda(), torch.from_numpy(s["start"]).cuda(),
                         torch.tensor(s["prefixes"], **i32), None, None, c, k,
                         kv_weight=s["kv_weight"].cuda(),
                         page_table=torch.from_numpy(s["table"]).cuda())
            # (another order of the norm's sum at another alignment: a last place of float32)
            tol = 2.0 ** -7 if dt is torch.bfloat16 else 2.0 ** -20
            for got, ref in ((c, want["c_kv"]), (k, want["k_pe"])):
                got = got.double().cpu().numpy()
                assert (np.abs(got - ref) <= tol * np.abs(ref) + 1e-30).all()
            rest = torch.cat([wide[:, :off], wide[:, off + 64:off + 72], wide[:, off + 88:]], -1)
            assert (rest == -77.0).all()


def test_starts_that_do_not_ascend():
    s = batch(78, [4, 4, 4], [5, 6, 7], 2, 16, 16, 64, torch.bfloat16)
    s["start"] = np.array([0, 9, 4, 12], np.int32)
    o = apply(s, status=tv.TV_ERR_BOUNDS)  # what it finds is anything, but within the arrays
    assert (o["q_pe"] == -77.0).any()


def test_captured_and_replayed():
    s = batch(76, [1] * 6, [3, 64, 127, 0, 900, 5], 16, 128, 64, 512, torch.bfloat16)
    want = apply(s)
    i32 = dict(dtype=torch.int32, device="cuda")
    out = {k: torch.zeros(v.shape, dtype=torch.bfloat16, device="cuda") for k, v in want.items()}
    prefix = torch.tensor([0] * 6, **i32)
    args = (s["q"].cuda(), s["kv"].cuda(), torch.from_numpy(s["start"]).cuda(), prefix,
            out["q_nope"], out["q_pe"], out["c_kv"], out["k_pe"])
    kw = dict(q_weight=s["q_weight"].cuda(), kv_weight=s["kv_weight"].cuda(),
              page_table=torch.from_numpy(s["table"]).cuda())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tv.norm_rope(*args, **kw)
    prefix.copy_(torch.tensor(s["prefixes"], **i32))
    for v in out.values():
        v.fill_(-77.0)
    graph.replay()
    torch.cuda.synchronize()
    for k in want:
        assert np.array_equal(out[k].double().cpu().numpy(), want[k])
