"""Outputs of the rotations that overlap what they are read from, or each other: refused (CPU: the
pointers are never followed), and slices between one another's rows are not (GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_decode_abi as abi
from tests import test_rope_any_gpu as ropes

BAD = tv.TV_ERR_INVALID_ARG
IN = abi.FAKE


@pytest.mark.parametrize("kw", [
    dict(out=IN + 4),                      # the next element, head, token
    dict(out=IN + 4 * 64), dict(out=IN - 4 * 64), dict(out=IN + 4 * 256), dict(out=IN - 4 * 256),
    dict(out=IN + 4 * (9 * 256 + 3 * 64 + 63)), dict(out=IN - 4 * (9 * 256 + 3 * 64 + 63)),
    # wider strides: heads that reach into the next slice's
    dict(out=IN + 4 * 63, in_stride_token=800, in_stride_head=200, out_stride_token=800,
         out_stride_head=200),
    dict(out=IN + 4 * 137, in_stride_token=800, in_stride_head=200, out_stride_token=800,
         out_stride_head=200),
    # heads outermost
    dict(out=IN + 4 * 64, in_stride_token=64, in_stride_head=640, out_stride_token=64,
         out_stride_head=640),
    # unequal strides: a token's heads meet; nothing to tell them by
    dict(out=IN + 4 * 255, in_stride_token=1000, out_stride_token=1000, out_stride_head=80),
    dict(out=IN + 4 * 700, in_stride_token=1000, out_stride_token=1000, out_stride_head=80),
    dict(out=IN + 4 * 300, in_stride_token=700, out_stride_token=900),
    # one vector for all tokens, in the middle of the output
    dict(out=IN - 4 * 1000, in_stride_token=0, in_stride_head=0),
])
def test_rope_refuses_an_overlapping_output(tvlib, kw):
    a = abi.rope_args(**kw)
    assert tv.load().tv_rope(ctypes.byref(a), None) == BAD
    assert b"overlap" in tv.load().tv_last_error()


CKV = abi.FAKE + 6 * abi.M


@pytest.mark.parametrize("kw", [
    dict(k_pe=CKV), dict(k_pe=CKV + 4 * 64), dict(k_pe=CKV + 4 * (1023 * 64 + 63)),
    dict(k_pe=CKV - 4 * 1023 * 16), dict(k_pe=CKV - 4 * 15),
    # slices of one buffer's rows that meet, of their own row or the next one
    dict(k_pe=CKV + 4 * 63, ckv_row_stride=80, kpe_row_stride=80),
    dict(k_pe=CKV + 4 * 65, ckv_row_stride=80, kpe_row_stride=80),
    dict(k_pe=CKV - 4 * 15, ckv_row_stride=80, kpe_row_stride=80),
    dict(k_pe=CKV + 4 * 130, ckv_row_stride=200, kpe_row_stride=100),
])
def test_norm_rope_refuses_cache_arrays_that_meet(tvlib, kw):
    a = abi.norm_args(**kw)
    assert tv.load().tv_norm_rope(ctypes.byref(a), None) == BAD
    assert b"overlap" in tv.load().tv_last_error()


def elements(start, token, head, T, H, d):
    return start + (np.arange(T)[:, None, None] * token + np.arange(H)[:, None] * head + np.arange(d))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_slices_of_one_buffer(tvlib, dt):
    r = np.random.default_rng(11)
    n = 12000
    taken = np.zeros(2, int)
    g = torch.Generator(device="cuda").manual_seed(12)
    for i in range(600):
        T, H, d = (int(v) for v in (r.integers(1, 6), r.integers(1, 5), 2 * r.integers(1, 33)))
        first, second = sorted(int(v) for v in r.integers(0, 140, 2))
        head = d + first
        token = (H - 1) * head + d + second
        if i % 3 == 1:                     # heads outermost
            token, head = d + first, (T - 1) * (d + first) + d + second
        strides = [(token, head), (token, head)]
        if i % 3 == 2:                     # another pitch of heads
            strides[1] = (token, int(r.integers(d, head + 1)))
        size = (T - 1) * token + (H - 1) * head + d
        a, b = 4000, 4000 + int(r.integers(-size, size + 1))
        if a == b:
            continue
        x, y = (elements(s, *st, T, H, d) for s, st in zip((a, b), strides))
        assert x.max() < n and 0 <= y.min() and y.max() < n
        buf = torch.randn(n, generator=g, device="cuda").to(dt)
        views = [buf.as_strided((T, H, d), (*st, 1), s) for s, st in zip((a, b), strides)]
        pos = torch.arange(T, dtype=torch.int32, device="cuda") + 9
        meet = len(np.intersect1d(x, y)) > 0
        if not meet:
            want = buf.clone()
            new = torch.empty((T, H, d), dtype=dt, device="cuda")
            tv.rope(views[0].contiguous(), new, pos)
            want.as_strided((T, H, d), (*strides[1], 1), b).copy_(new)
        try:
            tv.rope(views[0], views[1], pos)
        except tv.TVError as e:
            assert "overlap" in str(e)
            assert meet or strides[0] != strides[1]
            taken[0] += 1
            continue
        assert not meet
        assert torch.equal(buf, want)
        taken[1] += 1
    assert (taken > 100).all()


@pytest.mark.gpu
@pytest.mark.parametrize("at", [(0, 512), (64, 0), (8, 536), (80, 8)])
def test_cache_arrays_of_one_buffer(tvlib, at):
    s = ropes.batch(21, [5, 1, 70], [0, 63, 30], 2, 16, 64, 512, torch.bfloat16)
    want = ropes.apply(s)
    wide = torch.full((s["rows"], 600), -77.0, dtype=torch.bfloat16, device="cuda")
    c, k = wide[:, at[0]:at[0] + 512], wide[:, at[1]:at[1] + 64]
    tv.norm_rope(None, s["kv"].cuda(), torch.from_numpy(s["start"]).cuda(),
                 torch.tensor(s["prefixes"], dtype=torch.int32, device="cuda"), None, None, c, k,
                 kv_weight=s["kv_weight"].cuda(), page_table=torch.from_numpy(s["table"]).cuda())
    torch.cuda.synchronize()
    assert (c.double().cpu().numpy() == want["c_kv"]).all()
    assert (k.double().cpu().numpy() == want["k_pe"]).all()
