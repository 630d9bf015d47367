"""GPU tests of tv_prefill_attn (expanded-form latent attention) against its plain statement
in 64 bits.

Tolerance.  A rounding to bf16 is off by at most h = 2^-8 relative.  The kernel rounds the
expanded keys and the output to bf16, the expanded values and the softmax weights to fp16
(2^-11, counted as h here; everything else is 32-bit, below 1e-5 of it at these sizes).  With A = sum_j p_j |v_j| per output element, and
D = max_j scale sum_d |q_d k_jd| h the most a score moves (so that a weight moves by at most
e^(2D)), the output is within
    A (e^(2D) (1 + h)^2 - 1) + h |out| (1 + ..) + 1e-5 A.
That holds for every input.  For inputs of independent normal elements the four roundings are
independent, each of rms below h/sqrt(3) relative to what it rounds, and a score's error is of
rms below h/sqrt(3) * scale * sqrt(sum q^2 k^2), about 0.5 h for unit queries: the rms of a
row's error is then below 1.3 h of the row's rms at most, and 2 h = 2^-7 is asked of it.
"""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import serving_model as sm

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
H_STEP = 2.0 ** -8


def make(seed, H, lens, prefixes, DL=512, paged=True, q_scale=1.0, spare=2, tail=0):
    """A packed batch on the GPU; unused cache rows, and the workspace, hold NaN."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)

    def randn(*shape, s=1.0):
        return (torch.randn(shape, generator=g) * s).bfloat16()

    B, T = len(lens), sum(lens) + tail
    keys = [n + p if n else 0 for n, p in zip(lens, prefixes)]
    table, stride = None, 0
    if paged:
        need = [-(-k // 64) for k in keys]
        perm = r.permutation(sum(need) + spare)
        table = np.full((B, max(need) + 1), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        rows = len(perm) * 64
    else:
        stride = max(keys) + 3
        rows = B * stride
    c = torch.full((rows, DL), float("nan"), dtype=torch.bfloat16)
    k = torch.full((rows, 64), float("nan"), dtype=torch.bfloat16)
    s = dict(H=H, lens=lens, prefixes=prefixes, keys=keys, table=table, stride=stride,
             q_nope=randn(T, H, 128, s=q_scale), q_pe=randn(T, H, 64, s=q_scale),
             w_kv=randn(H, 256, DL, s=DL ** -0.5), scale=192 ** -0.5, rows=[])
    for b in range(B):
        j = np.arange(keys[b])
        at = (table[b, j // 64].astype(np.int64) * 64 + j % 64) if paged else b * stride + j
        s["rows"].append(torch.from_numpy(at))
        c[at], k[at] = randn(keys[b], DL), randn(keys[b], 64)
    s["c_kv"], s["k_pe"] = c, k
    s["start"] = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return s


def device(s):
    d = {k: v.cuda() for k, v in s.items() if isinstance(v, torch.Tensor)}
    d["table"] = None if s["table"] is None else torch.from_numpy(s["table"]).cuda()
    d["start"] = torch.from_numpy(s["start"]).cuda()
    d["prefix"] = torch.tensor(s["prefixes"], dtype=torch.int32, device="cuda")
    d["out"] = torch.full((*s["q_nope"].shape[:2], 128), -77.0, dtype=torch.bfloat16,
                          device="cuda")
    d["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return d


def launch(s, d, **kw):
    p = dict(max_q_len=max(s["lens"]), max_kv_len=max(s["keys"]), total_kv=sum(s["keys"]),
             page_table=d["table"], kv_stride_b=s["stride"], status=d["status"])
    p.update(kw)
    tv.prefill_attn(d["q_nope"], d["q_pe"], d["w_kv"], d["c_kv"], d["k_pe"], d["start"],
                    d["prefix"], d["out"], s["scale"], **p)


def workspace(s, d):
    a = tv.prefill_args(d["q_nope"], d["q_pe"], d["w_kv"], d["c_kv"], d["k_pe"], d["start"],
                        d["prefix"], d["out"], s["scale"], max(s["lens"]), max(s["keys"]),
                        sum(s["keys"]), d["table"], 64, s["stride"])
    return torch.full((tv.prefill_workspace_size(a),), 255, dtype=torch.uint8, device="cuda")


def run(s, status=0, **kw):
    d = device(s)
    launch(s, d, workspace=workspace(s, d), **kw)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == status
    return d["out"].double().cpu().numpy()


def close(s, out, b, rms=True):
    """Sequence b of the output against the plain statement, by both rules."""
    lo, n = int(s["start"][b]), s["lens"][b]
    q, qp = (s[k][lo:lo + n].double().numpy() for k in ("q_nope", "q_pe"))
    w = s["w_kv"].double().numpy()
    c, kp = (s[k][s["rows"][b]].double().numpy() for k in ("c_kv", "k_pe"))
    ref = sm.prefill(q, qp, w, c, kp, s["prefixes"][b], s["scale"])
    got = out[lo:lo + n]
    assert np.isfinite(got).all()
    hidden = np.arange(len(c))[None] > s["prefixes"][b] + np.arange(n)[:, None]
    for h in range(s["H"]):
        kv = c @ w[h].T
        k, v = kv[:, :128], kv[:, 128:]
        x = (q[:, h] @ k.T + qp[:, h] @ kp.T) * s["scale"]
        x[hidden] = -np.inf
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        A = p @ np.abs(v)
        moved = np.abs(q[:, h]) @ np.abs(k).T * s["scale"] * H_STEP
        moved[hidden] = 0
        D = moved.max(1, keepdims=True)
        tol = (A * (np.exp(2 * D) * (1 + H_STEP) ** 2 - 1 + 1e-5)) * (1 + H_STEP) \
            + H_STEP * np.abs(ref[:, h]) + 1e-6
        assert (np.abs(got[:, h] - ref[:, h]) <= tol).all(), (b, h)
    if rms:
        e = np.sqrt(((got - ref) ** 2).mean(-1)) / np.sqrt((ref ** 2).mean(-1))
        assert e.max() <= 2 * H_STEP, (b, e.max())


def check(s, **kw):
    out = run(s)
    for b in range(len(s["lens"])):
        if s["lens"][b]:
            close(s, out, b, **kw)
    return out


@pytest.mark.parametrize("n", [1, 2, 33, 127, 128, 129, 255, 256, 257, 300, 640])
@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 129])
def test_lengths(n, prefix):
    """Every way a tile, a key block and a page can end."""
    check(make(n * 7 + prefix, 2, [n], [prefix], DL=128, paged=prefix % 2 == 1))


@pytest.mark.parametrize("H,DL", [(1, 64), (3, 512), (5, 192), (16, 512), (64, 512)])
def test_heads_and_latent_sizes(H, DL):
    check(make(H, H, [70], [40], DL=DL))


@pytest.mark.parametrize("paged", [True, False])
def test_ragged_batch(paged):
    """Prompts, chunks after a prefix, single tokens and empty sequences; rows behind the
    last sequence stay as they were."""
    s = make(3, 3, [1, 200, 0, 33, 513, 0, 128, 1], [700, 0, 50, 257, 64, 0, 900, 0],
             DL=128, paged=paged, tail=9)
    out = check(s)
    assert (out[s["start"][-1]:] == -77).all()


def test_more_sequences_than_a_block_has_threads():
    s = make(4, 1, [1] * 1500, [i % 5 for i in range(1500)], DL=64)
    out = run(s)
    for b in (0, 1, 1023, 1024, 1025, 1499):
        close(s, out, b)


def test_long_prompt_sampled_rows():
    """4096 keys, 8 heads: rows of every tile against one-row calls of the statement."""
    s = make(5, 8, [4096], [0])
    out = run(s)
    for i in (0, 1, 127, 128, 255, 256, 2047, 3000, 4095):
        one = dict(s, lens=[1], prefixes=[i], start=np.array([i, i + 1]),
                   rows=[s["rows"][0][:i + 1]])
        close(one, out, 0)


@pytest.mark.parametrize("H", [1, 2, 5])
@pytest.mark.parametrize("prefix", [1100, 5000])
def test_few_items_are_cut_along_the_keys(H, prefix):
    """A batch that leaves SMs idle: up to 38 pieces of an item, some of a short sequence
    empty, some beginning at the diagonal with all their keys hidden from the first rows."""
    check(make(19 + H, H, [256, 200, 1, 129, 300], [prefix, 100, 0, 200, 900], DL=64))


@pytest.mark.parametrize("H,lens,prefixes", [
    (50, [130, 5], [1500, 3]),                     # one tile in two pieces, one written at once
    (16, [256, 256, 256, 256], [6000, 3840, 2048, 511]),
    (75, [129, 7], [700, 700]),                    # two pieces in all: nothing is cut
])
def test_cut_and_whole_tiles_side_by_side(H, lens, prefixes):
    out = check(make(24, H, lens, prefixes, DL=64))
    assert np.array_equal(run(make(24, H, lens, prefixes, DL=64)), out)


def test_cut_items_rescale_and_repeat():
    s = make(21, 2, [140], [2500], DL=64, q_scale=8.0)
    ramp = torch.linspace(0.1, 2, 2640)[:, None]
    s["c_kv"][s["rows"][0]] = (s["c_kv"][s["rows"][0]].float() * ramp).bfloat16()
    out = check(s, rms=False)
    assert np.array_equal(run(s), out)


def test_sharp_softmax():
    s = make(6, 2, [300], [100], DL=128, q_scale=12.0)
    check(s, rms=False)


def test_rising_scores_rescale():
    """Keys grow along the sequence, so that the running maximum keeps moving."""
    s = make(7, 2, [260], [390], DL=128)
    s["q_nope"] = s["q_nope"].abs()
    s["w_kv"][:, :128] = s["w_kv"][:, :128].abs()
    ramp = torch.linspace(0, 4, 650)[:, None]
    s["c_kv"][s["rows"][0]] = (s["c_kv"][s["rows"][0]].float().abs() * ramp).bfloat16()
    check(s, rms=False)
    s["c_kv"] = -s["c_kv"]  # and falls
    check(s, rms=False)


def test_strided_cache_rows():
    s = make(8, 2, [150], [20], DL=128)
    e = run(s)
    d = device(s)
    c = torch.full((d["c_kv"].shape[0], 200), float("nan"), dtype=torch.bfloat16, device="cuda")
    k = torch.full((d["k_pe"].shape[0], 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    c[:, 8:136], k[:, 8:72] = d["c_kv"], d["k_pe"]
    d["c_kv"], d["k_pe"] = c[:, 8:136], k[:, 8:72]
    launch(s, d)
    torch.cuda.synchronize()
    assert np.array_equal(d["out"].double().cpu().numpy(), e)


def test_repeated_calls_give_the_same_bits():
    s = make(9, 4, [400, 90], [33, 800])
    assert np.array_equal(run(s), run(s))


@pytest.mark.parametrize("what", ["negative", "descending", "past_T", "prefix", "q_len",
                                  "kv_len", "total"])
def test_bad_sequences_are_left_out(what):
    s = make(10, 2, [40, 60, 50], [5, 6, 7], DL=128)
    good = run(s)
    t, kw, bad = dict(s), {}, [1]
    t["start"] = s["start"].copy()
    if what == "negative":
        t["start"][0], bad = -1, [0]
    elif what == "descending":
        t["start"] = np.array([0, 40, 30, 80], np.int32)
        bad = [1, 2]
    elif what == "past_T":
        t["start"][3], bad = 151, [2]
    elif what == "prefix":
        t["prefixes"] = [5, -6, 7]
    elif what == "q_len":
        kw = dict(max_q_len=59)
    elif what == "kv_len":
        kw = dict(max_kv_len=65)
    else:  # room for the first two only: the padding of three sequences is not in it
        kw, bad = dict(total_kv=1), []
    d = device(t)
    launch(t, d, **kw)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == (0 if what == "total" else tv.TV_ERR_BOUNDS)
    out = d["out"].double().cpu().numpy()
    for b in range(3):
        rows = slice(int(s["start"][b]), int(s["start"][b + 1]))
        assert np.array_equal(out[rows], good[rows] if b not in bad
                              else np.full_like(good[rows], -77))


def test_more_keys_than_announced():
    s = make(11, 1, [300, 300, 300], [0, 0, 0], DL=64)
    d = device(s)
    launch(s, d, total_kv=500)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == tv.TV_ERR_BOUNDS
    out = d["out"].double().cpu().numpy()
    close(s, out, 0)
    close(s, out, 1)
    assert (out[600:] == -77).all()


@pytest.mark.parametrize("page", [-1, 10 ** 6, 2 ** 31 - 1])
def test_pages_outside_the_cache_read_as_zeros(page):
    s = make(12, 2, [100], [60], DL=128)
    s["table"][0, 1] = page
    out = run(s, tv.TV_ERR_BOUNDS)
    for k in ("c_kv", "k_pe"):  # the statement: that page's rows are zero
        s[k] = torch.cat([s[k], torch.zeros((1, s[k].shape[1]), dtype=torch.bfloat16)])
    s["rows"][0][64:128] = len(s["c_kv"]) - 1
    close(s, out, 0, rms=False)


def test_values_past_the_fp16_range_are_clamped_and_reported():
    s = make(18, 2, [40], [100], DL=64)
    s["w_kv"][1, 128 + 5] = 512.0
    s["c_kv"][s["rows"][0][77]] = 4.0      # 64 * 4 * 512 = 131072
    out = run(s, tv.TV_ERR_BOUNDS)
    one = dict(s, H=1, q_nope=s["q_nope"][:, :1], q_pe=s["q_pe"][:, :1], w_kv=s["w_kv"][:1])
    close(one, out[:, :1], 0, rms=False)   # the other head is untouched
    assert np.isfinite(out).all() and out[:, 1, 5].max() <= 65504
    s["c_kv"][s["rows"][0][77]] = 1.9921875  # 65280: in range
    run(s)


def test_captured_and_replayed_with_other_lengths():
    a = make(13, 2, [200, 57], [30, 400], DL=128)
    b = make(14, 2, [57, 130], [200, 1], DL=128)
    d = device(a)
    T = 257
    bounds = dict(max_q_len=256, max_kv_len=512, total_kv=1024)
    table = torch.full((2, 12), -1, dtype=torch.int32, device="cuda")
    table[:, :a["table"].shape[1]] = d["table"]
    d["table"] = table
    c, k = (torch.zeros((40 * 64, n), dtype=torch.bfloat16, device="cuda") for n in (128, 64))
    c[:len(a["c_kv"])], k[:len(a["k_pe"])] = d["c_kv"], d["k_pe"]
    d["c_kv"], d["k_pe"] = c, k
    launch(a, d, **bounds)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        launch(a, d, **bounds)
    for s in (b, a):
        e = device(s)
        for name in ("q_nope", "q_pe", "w_kv", "c_kv", "k_pe"):
            d[name][:len(e[name])].copy_(e[name])
        table.fill_(-1)
        table[:, :e["table"].shape[1]].copy_(e["table"])
        d["start"].copy_(e["start"])
        d["prefix"].copy_(e["prefix"])
        g.replay()
        torch.cuda.synchronize()
        assert int(d["status"].item()) == 0
        out = d["out"].double().cpu().numpy()
        for i in range(2):
            close(s, out, i)
    assert T >= sum(b["lens"])


def test_two_streams_at_once():
    s = [make(15 + i, 4, [300, 20], [100, 700], DL=128) for i in range(2)]
    d = [device(x) for x in s]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    for _ in range(4):
        for x, y, st in zip(s, d, streams):
            launch(x, y, stream=st)
    torch.cuda.synchronize()
    for x, y in zip(s, d):
        for b in range(2):
            close(x, y["out"].double().cpu().numpy(), b)


def test_agrees_with_the_absorbed_form():
    """tv_verify_attn under the causal mask on q_nope W_uk, with W_uv applied to its output:
    the two forms differ by the roundings of both (each within 2^-7 of a row's rms, and the
    absorbed query's own rounding within 2^-8 of the scores)."""
    H, n, P = 8, 200, 150
    s = make(17, H, [n], [P], paged=False)
    out = run(s)
    d = device(s)
    for k in ("c_kv", "k_pe"):  # the absorbed kernel weighs rows behind the keys with zero
        d[k] = d[k].nan_to_num()
    w = d["w_kv"].float()
    ql = torch.einsum("thd,hdl->thl", d["q_nope"].float(), w[:, :128]).bfloat16()[None]
    lat = torch.empty((1, n, H, 512), device="cuda")
    lse = torch.empty((1, n, H), device="cuda")
    tv.verify_attn(ql.contiguous(), d["q_pe"][None], d["c_kv"], d["k_pe"], d["prefix"], None,
                   lat, lse, s["scale"], P, kv_stride_b=s["stride"], mask_mode=tv.MASK_CAUSAL)
    ref = torch.einsum("thl,hvl->thv", lat[0], w[:, 128:]).double().cpu().numpy()
    e = np.sqrt(((out - ref) ** 2).mean(-1)) / np.sqrt((ref ** 2).mean(-1))
    assert e.max() <= 2.0 ** -6, e.max()
