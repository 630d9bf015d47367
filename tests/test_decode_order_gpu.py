"""GPU tests of what stands before and behind a tv_shared_attn call on its stream, with no
synchronisation in between: its outputs are read, its queries written anew and its workspace used by
the next call, bit for bit as when every call is waited for.

Short sequences that are not swept together are written by the attention kernel itself, so that
nothing is left to join; the last batch of each list has partial results."""
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv
from tests import test_shared_attn_gpu as shared

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
BATCHES = [
    dict(members=[1], shared=[0], own=[299]),
    dict(members=[4], shared=[200], own=[50, 51, 52, 53]),
    dict(members=[40], shared=[0], own=370, H=64),
    dict(members=[3], shared=[0], own=[60, 0, 130], H=5, Q=9),
    dict(members=[6], shared=[1280], own=60),
]


def batch(seed, kw):
    """A batch with its queries' unrotated rope parts, two passes' worth of them."""
    s = shared.make(seed, **kw)
    d = shared.device(s)
    g = torch.Generator(device="cuda").manual_seed(seed)
    d["raw"] = torch.randn((2, s["B"] * s["Q"], s["H"], 64), generator=g, device="cuda").bfloat16()
    d["q_start"] = torch.arange(s["B"] + 1, dtype=torch.int32, device="cuda") * s["Q"]
    return s, d


def turn_queries(s, d, i):
    """The queries of pass i, by a kernel that may start before the one ahead of it has ended."""
    T = s["B"] * s["Q"]
    tv.norm_rope(d["raw"][i], None, d["q_start"], d["prefix"], None,
                 d["q_pe"].view(T, s["H"], 64), None, None, status=d["status"])


def passes(batches, workspace, between, wait=lambda: None):
    """Two passes over the batches on one workspace; what every call has written, as it stood."""
    seen = []
    for i in range(2):
        for s, d in batches:
            turn_queries(s, d, i)
            wait()
            shared.launch(s, d, workspace=workspace)
            wait()
            if between == "queries":      # written again right behind
                turn_queries(s, d, 1 - i)
                wait()
            if between != "calls":        # (else the next call comes first)
                seen.append((d["out"].clone(), d["lse"].clone()))
                wait()
        if between == "calls":
            seen += [(d["out"].clone(), d["lse"].clone()) for _, d in batches]
            wait()
    return seen


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("between", ["queries", "outputs", "calls"])
def test_no_call_comes_too_early(between, captured):
    batches = [batch(300 + i, kw) for i, kw in enumerate(BATCHES)]
    size = max(len(shared.poisoned_workspace(s, d)) for s, d in batches)
    workspace = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    want = passes(batches, workspace, between, torch.cuda.synchronize)
    assert all(int(d["status"].item()) == 0 for _, d in batches)
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = passes(batches, workspace, between)
        play = graph.replay
    else:
        got = []

        def play():
            got[:] = passes(batches, workspace, between)
    for _ in range(20):
        for _, d in batches:
            d["out"].fill_(-77.0)
            d["lse"].fill_(-77.0)
        play()
        torch.cuda.synchronize()
        for (out, lse), (o, l) in zip(got, want, strict=True):
            assert torch.equal(out, o) and torch.equal(lse, l)


def test_the_synchronised_results_are_right():
    for i, kw in enumerate(BATCHES):
        s, d = batch(300 + i, kw)
        turn_queries(s, d, 0)
        torch.cuda.synchronize()
        shared.launch(s, d)
        torch.cuda.synchronize()
        shared.close(s, d)
