"""GPU tests of tv_prefill_attn where it can go wrong: bounds at the ends of their range, NaN
in cut items, weights far below a row's largest, running maxima that move.

The roundings that the tolerances count are those of tests/test_prefill_attn_gpu.py."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_prefill_attn_gpu as base

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("where", [0, 1])
def test_a_prefix_at_the_end_of_the_integers(where):
    """Host bounds without a limit and a prefix of nearly 2^31 keys: the sequence has more
    blocks of keys than were announced, so it and those behind it are left out."""
    s = base.make(31, 1, [40, 40], [5, 5], DL=64, paged=False)
    good = base.run(s)
    s["prefixes"][where] = INT_MAX - 40
    d = base.device(s)
    base.launch(s, d, max_kv_len=INT_MAX, total_kv=90, kv_stride_b=INT_MAX)
    torch.cuda.synchronize()
    assert int(d["status"].item()) == tv.TV_ERR_BOUNDS
    out = d["out"].double().cpu().numpy()
    done = 40 * where
    assert np.array_equal(out[:done], good[:done]) and (out[done:] == -77).all()
