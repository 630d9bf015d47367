"""GPU tests of tv_shared_attn with many rows, where a warp of its join takes more than one part of
the columns: rows in one piece, rows to be joined and rows of sequences out of bounds beside each
other.  Tolerance as in test_shared_attn_gpu.py."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_shared_attn_gpu as shared

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]


def test_all_rows_joined():
    s = shared.make(401, [40], [1280], 60, H=128, Q=5)
    shared.close(s, shared.run(s), sequences=[0, 17, 39])


@pytest.mark.parametrize("Q,out", [(5, torch.float32), (64, torch.bfloat16)])
def test_rows_of_every_kind(Q, out):
    # two sequences alone of few keys, a group swept together, one cut along its keys, one out of
    # bounds, and more alone: 102400 or 819200 rows as a whole
    B, H = (160, 128) if Q == 5 else (100, 128)
    members, keys = [1, 1, 3, 1, 1] + [1] * (B - 7), [64, 300, 1500, 9000, 100]
    keys += [70 + b % 190 for b in range(B - 7)]
    start = np.concatenate([[0], np.cumsum(members)])
    group = np.repeat(np.arange(len(members)), members)
    prefix = np.array([keys[i] for i in group])
    common = [1472 if i == 2 else 0 for i in range(len(members))]
    need = -(-(prefix + Q) // 64)
    table = np.full((B, int(need.max())), -1, np.int32)
    at = 0
    for b in range(B):
        first = common[group[b]] // 64 if start[group[b]] != b else 0
        table[b, :first] = table[start[group[b]], :first]
        table[b, first:need[b]] = at + np.arange(need[b] - first)
        at += need[b] - first
    g = torch.Generator(device="cuda").manual_seed(402)

    def randn(*shape, s=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * s).bfloat16()

    def put(a):
        return torch.from_numpy(np.asarray(a, np.int32)).cuda()
    c, k = randn(at * 64, 512), randn(at * 64, 64)
    ql, qp = randn(B, Q, H, 512, s=0.25), randn(B, Q, H, 64)
    rows = [np.repeat(table[b], 64)[:prefix[b] + Q].astype(np.int64) * 64 +
            np.arange(prefix[b] + Q) % 64 for b in range(B)]
    told = prefix.copy()
    told[6] = -1
    o = torch.full((B, Q, H, 512), -77.0, dtype=out, device="cuda")
    lse = torch.full((B, Q, H), -77.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tv.shared_attn(ql, qp, c, k, put(told), put(start), put(common), o, lse, 192 ** -0.5,
                   max_prefix_len=9000, page_table=put(table), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == tv.TV_ERR_BOUNDS
    assert (o[6] == 0).all() and (lse[6] == -math.inf).all()
    s = dict(Q=Q, B=B, H=H, scale=192 ** -0.5, vis=np.tri(Q, dtype=bool)[None].repeat(B, 0),
             keys=[(c[r], k[r]) for r in rows])
    d = dict(q_latent=ql, q_pe=qp, out=o, lse=lse)
    for b in (0, 1, 2, 4, 5, 7, 60, B - 1):
        at = slice(0, 8) if Q == 64 else slice(0, Q)      # (the first rows, all heads)
        if Q == 5:
            shared.close(s, d, [b])
            continue
        n = len(rows[b]) - Q + 8                          # the keys that those see
        part = dict(s, Q=8, vis=np.tri(8, dtype=bool)[None].repeat(B, 0),
                    keys=[(x[:n], y[:n]) if i == b else None for i, (x, y) in enumerate(s["keys"])])
        shared.close(part, {name: t[:, at] for name, t in d.items()}, [b])
