"""Bounded waits of the prompt kernels: a producer that stops issuing loads, without any fault,
makes the waits of the others run out, and the kernels give up cleanly.

With the deadline at 10 ms and the producer of every CTA stopped after a number of loads
(before the first, in the middle of a tile or of the ring, between a block's keys and its
values), expected are TV_ERR_TIMEOUT, that every CTA leaves, those with work left through the
abort path, and that a following normal call is correct to the bit, which it could not be if
tensor memory had been left allocated or a copy still in flight."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_prefill_attn_gpu as base


@contextlib.contextmanager
def fault(expand, attend, counts):
    lib = tv.load()
    assert lib.tv_testing_set_prompt_fault(expand, attend, 10_000_000,
                                           ctypes.c_void_p(counts.data_ptr())) == tv.TV_OK
    try:
        yield
    finally:
        assert lib.tv_testing_set_prompt_fault(-1, -1, 0, None) == tv.TV_OK


# (the hook's own limits, on CPU)
def test_hook_rejects_a_long_deadline(tvlib):
    lib = tv.load()
    assert lib.tv_testing_set_prompt_fault(-1, -1, 2_000_000_001, None) == tv.TV_ERR_INVALID_ARG
    assert lib.tv_testing_set_prompt_fault(-1, -1, 0, None) == tv.TV_OK


WHOLE = dict(H=80, lens=[200, 200], prefixes=[600, 700])  # 1200 tiles, 160 items: work everywhere
CUT = dict(H=1, lens=[200], prefixes=[1500])              # 14 tiles, one item in 4 pieces


@pytest.mark.parametrize("case,expand,attend", [
    (WHOLE, 0, -1), (WHOLE, 5, -1), (WHOLE, 13, -1), (CUT, 0, -1), (CUT, 5, -1),
    (WHOLE, -1, 0), (WHOLE, -1, 1), (WHOLE, -1, 2), (WHOLE, -1, 3), (WHOLE, -1, 6),
    (CUT, -1, 0), (CUT, -1, 1), (CUT, -1, 2), (CUT, -1, 5), (WHOLE, 3, 3)])
@pytest.mark.gpu
def test_waits_run_out_and_the_next_call_is_correct(tvlib, case, expand, attend):
    s = base.make(51, DL=512, **case)
    d = base.device(s)
    ws = base.workspace(s, d)
    ws.zero_()
    base.launch(s, d, workspace=ws)
    torch.cuda.synchronize()
    good = d["out"].clone()
    assert int(d["status"].item()) == 0
    counts = torch.zeros(4, dtype=torch.int32, device="cuda")
    with fault(expand, attend, counts):
        base.launch(s, d, workspace=ws)
        torch.cuda.synchronize()
    assert int(d["status"].item()) == tv.TV_ERR_TIMEOUT
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    whole = case is WHOLE
    e_left, e_gave, a_left, a_gave = counts.tolist()
    assert e_left == (sms if whole else 15) and a_left == sms
    assert e_gave == (0 if expand < 0 else sms if whole else 14)
    assert a_gave == (0 if attend < 0 else sms if whole else 4)
    # the same stream and buffers: a normal call now
    d["status"].zero_()
    d["out"].fill_(float("nan"))
    base.launch(s, d, workspace=ws)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == 0 and torch.equal(d["out"], good)
    out = good.double().cpu().numpy()
    base.close(dict(s, H=1, q_nope=s["q_nope"][:, :1], q_pe=s["q_pe"][:, :1], w_kv=s["w_kv"][:1]),
               out[:, :1], 0)
    assert np.isfinite(out).all()
