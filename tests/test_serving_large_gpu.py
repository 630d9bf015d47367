"""GPU tests of the serving calls at the far end of what they take: pools whose page counts no
longer fit in a thread's bits, 4096 rows, offsets past 2^31 elements, long prefixes, and the
block sizes of the sampling kernel that the other tests do not reach."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import serving_model as sm
from tests import test_prefill_attn_gpu as prompts
from tests.test_pages_gpu import Both
from tests.test_sample_gpu import call, check, make

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]


@pytest.mark.parametrize("num", [8 * 1024 * 64, 8 * 1024 * 64 + 1, 1_000_003])
def test_pools_of_more_pages_than_bits(num):
    """A thread's run of pages is 64 long, one longer, and twice that."""
    rows, most, ps = 9, 40_000, 1
    b = Both(rows, most, num, ps)
    r = np.random.default_rng(num)
    length = r.integers(20_000, 39_000, rows)
    perm, at = r.permutation(num), 0                  # pages all over the pool
    for k in range(rows):
        b.m.table[k, :length[k]] = perm[at:at + length[k]]
        b.m.ref[perm[at:at + length[k]]] = 1
        b.m.n[k] = length[k]
        at += length[k]
    b.upload()
    gone = np.where(np.arange(rows) % 3 == 1, 0, np.where(np.arange(rows) % 3 == 2, length // 2, -1))
    b.release(gone)
    length = np.where(gone >= 0, gone, length)
    src = np.full(rows, -1)
    src[1], length[1] = 0, length[0] - 3
    b.fork(src, length)
    new = np.minimum(length + r.integers(0, 500, rows), most)
    b.reserve(length, new)
    c = b.compact()
    assert len(c) > 1000
    length = np.maximum(length, new)
    b.reserve(length, np.minimum(length + 300, most))
    b.m.check()


def test_four_thousand_rows():
    rows, num, ps = 4096, 40_000, 16
    b = Both(rows, 12, num, ps)
    r = np.random.default_rng(3)
    length = r.integers(0, 60, rows)
    b.reserve([0] * rows, length)
    half = np.arange(rows) >= rows // 2
    b.release(np.where(half, 0, -1))
    src = np.where(half, r.integers(0, rows // 2, rows), -1)
    length = np.where(half, length[np.maximum(src, 0)], length)
    b.fork(src, length)
    c = b.reserve(length, length + r.integers(0, 40, rows))
    assert (c[:, 0] >= 0).sum() > 500
    b.compact()
    b.m.check()


@pytest.mark.parametrize("draft", [None, "depth"])
@pytest.mark.parametrize("B,V,dtype", [(12, 70001, "fp32"), (17, 66000, "bf16"), (9, 131000, "bf16"),
                                       (1, 163840, "fp32")])
def test_larger_blocks(B, V, dtype, draft):
    """Clusters of 16 CTAs of 512 threads, and of 1024."""
    check(make(B + V, B, 6, V, dtype, draft))


def test_logits_and_drafter_rows_past_2_31_elements():
    """The last sequences of a large batch, against a call of their own."""
    B, Q, V = 134, 64, 1 << 18
    small = make(91, 2, Q, V, "bf16", "node", spread=1.0)
    want, status = call(small)
    assert status == 0
    logits = torch.zeros((B, Q, V), dtype=torch.bfloat16, device="cuda")
    draft = torch.zeros((B, Q, V), device="cuda")
    s = {k: torch.zeros((B, *v.shape[1:]), dtype=v.dtype) for k, v in small.items()
         if isinstance(v, torch.Tensor) and k not in ("logits", "draft")}
    s["parent"][:] = small["parent"][:1]
    s["tokens"][:] = -1                               # (the others test nothing)
    for k in s:
        s[k][-2:] = small[k]
    logits[-2:], draft[-2:] = small["logits"].cuda(), small["draft"].cuda()
    got, status = call(dict(s, logits=logits, draft=draft, by_node=True))
    assert status == 0
    for g, w in zip(got, want):
        assert np.array_equal(g[-2:], w)


@pytest.mark.parametrize("H,DL", [(1, 64), (2, 1088)])
def test_long_prefixes(H, DL):
    s = prompts.make(92, H, [3, 130], [131_000, 40], DL=DL)
    prompts.check(s)


def test_cache_rows_and_expanded_keys_past_2_31_elements(monkeypatch):
    """The same prompt in the first pages of a small cache and in the last of one of 4.3 million
    rows, and its last heads where their expanded keys lie past 2^31 elements."""
    monkeypatch.setattr(tv, "_ws_cache", {})          # 11 GB that no other test needs
    H, DL, n, P = 2, 512, 140, 300
    s = prompts.make(93, H, [n], [P], DL=DL)
    want = prompts.run(s)
    d = prompts.device(s)
    pages = s["table"].shape[1] - 1
    rows = 4_300_032
    c = torch.zeros((rows, DL), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    table = np.full_like(s["table"], -1)
    for i in range(pages):
        page = rows // 64 - 1 - 3 * i
        old = int(s["table"][0, i])
        c[page * 64:page * 64 + 64] = d["c_kv"][old * 64:old * 64 + 64]
        k[page * 64:page * 64 + 64] = d["k_pe"][old * 64:old * 64 + 64]
        table[0, i] = page
    d["c_kv"], d["k_pe"], d["table"] = c, k, torch.from_numpy(table).cuda()
    prompts.launch(s, d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    assert np.array_equal(d["out"].double().cpu().numpy(), want)
    # 160 heads with room for 132000 keys: 2.7 * 10^9 elements of keys; heads repeat the two
    for name in ("q_nope", "q_pe", "w_kv"):
        axis = 0 if name == "w_kv" else 1
        d[name] = torch.cat([d[name]] * 80, axis).contiguous()
    d["out"] = torch.zeros((n, 160, 128), dtype=torch.bfloat16, device="cuda")
    prompts.launch(s, d, total_kv=132_000)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    out = d["out"].double().cpu().numpy()
    # (whole items here, cut ones above: equal but for the order of sums and one rounding)
    assert np.array_equal(out[:, :2], out[:, -2:])
    prompts.close(s, out[:, :2], 0)
