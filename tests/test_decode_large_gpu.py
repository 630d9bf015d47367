"""GPU tests of the decode calls past 2^31 elements: caches, logits and heads far apart, each
against the same call on its small copy."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_rope_any_gpu as ropes
from tests import test_shared_attn_gpu as shared
from tests import test_token_gpu as tokens

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
ROWS = 4_300_032  # x 512 elements: past 2^31; pages of 64


def big(d):
    return torch.empty((ROWS, d), dtype=torch.bfloat16, device="cuda")


def test_shared_attention_at_the_end_of_a_long_cache():
    s = shared.make(91, [5, 2], [1280, 300], 70, Q=2)
    want, d = shared.run(s), shared.device(s)
    small = len(s["c_kv"])
    d["c_kv"], d["k_pe"] = big(512), big(64)
    d["c_kv"][-small:], d["k_pe"][-small:] = s["c_kv"].cuda(), s["k_pe"].cuda()
    d["table"] = torch.where(d["table"] < 0, -1, d["table"] + (ROWS - small) // 64)
    shared.launch(s, d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    assert torch.equal(d["out"], want["out"]) and torch.equal(d["lse"], want["lse"])


def test_shared_attention_of_sequences_far_apart():
    s = shared.make(92, [2], [640], 70, paged=False)
    want, d = shared.run(s), shared.device(s)
    n, old = s["stride"], s["stride"]
    s["stride"] = ROWS // 2
    d["c_kv"], d["k_pe"] = big(512), big(64)
    for b in range(2):
        for name in ("c_kv", "k_pe"):
            d[name][b * (ROWS // 2):][:n] = s[name][b * old:][:n].cuda()
    shared.launch(s, d)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0
    assert torch.equal(d["out"], want["out"]) and torch.equal(d["lse"], want["lse"])


@pytest.mark.parametrize("paged", [True, False])
def test_keys_into_a_long_cache(paged):
    s = ropes.batch(93, [5, 70], [100, 3], 2, 16, 64, 512, torch.bfloat16, paged=paged)
    want = ropes.apply(s)
    c, k = big(512), big(64)
    table, stride = None, 0
    at = np.arange(s["rows"])
    if paged:
        move = ROWS // 64 - s["rows"] // 64
        table = torch.from_numpy(np.where(s["table"] < 0, -1, s["table"] + move)).cuda()
        at = at + move * 64
    else:
        stride = ROWS // 2
        at = at // s["stride"] * stride + at % s["stride"]
    at = torch.from_numpy(at).cuda()
    c[at], k[at] = -77.0, -77.0
    i32 = dict(dtype=torch.int32, device="cuda")
    tv.norm_rope(None, s["kv"].cuda(), torch.from_numpy(s["start"]).cuda(),
                 torch.tensor(s["prefixes"], **i32), None, None, c, k,
                 kv_weight=s["kv_weight"].cuda(), page_table=table, kv_stride_b=stride)
    torch.cuda.synchronize()
    assert (c[at].double().cpu().numpy() == want["c_kv"]).all()
    assert (k[at].double().cpu().numpy() == want["k_pe"]).all()


def test_heads_far_apart():
    T, H, D, far = 3, 2, 64, 1_100_000_008
    g = torch.Generator(device="cuda").manual_seed(94)
    x = torch.randn((T, H, D), generator=g, device="cuda").bfloat16()
    pos = torch.tensor([5, 70, 900], dtype=torch.int32, device="cuda")
    want = torch.empty_like(x)
    tv.rope(x, want, pos)
    wide = torch.empty(2 * far + H * D, dtype=torch.bfloat16, device="cuda")
    v = wide.as_strided((T, H, D), (far, D, 1))
    v.copy_(x)
    tv.rope(v, v, pos)
    torch.cuda.synchronize()
    assert torch.equal(v, want)


def test_logits_far_apart():
    logits, u = tokens.rows(95, 3, 5003, torch.bfloat16)
    far = 1_100_000_007
    wide = torch.empty(2 * far + 5003, dtype=torch.bfloat16, device="cuda")
    v = wide.as_strided((3, 5003), (far, 1))
    v.copy_(logits)
    for kw in (dict(), dict(k=40), dict(p=0.9)):
        got, want = tokens.sample(v, u, **kw), tokens.sample(logits.cuda(), u, **kw)
        assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


def test_what_may_be_left_out():
    logits, u = tokens.rows(96, 5, 700)
    t = torch.full((5,), -9, dtype=torch.int32, device="cuda")
    tv.token_sample(logits.cuda(), torch.from_numpy(u).cuda(), t)
    assert t.tolist() == tokens.sample(logits.cuda(), u)[0].tolist()
    s = shared.make(97, [4], [640], 50, tree=False)
    want, d = shared.run(s), shared.device(s)
    shared.launch(s, d, status=None, lse=None)
    torch.cuda.synchronize()
    assert torch.equal(d["out"], want["out"]) and (d["lse"] == -77.0).all()
