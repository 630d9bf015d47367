"""The binding's workspaces: whose device and stream they belong to (no GPU needed: the CUDA
calls are stood in for)."""
import contextlib

import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv


class FakeCuda:
    """Current device and stream, and where each allocation was made."""

    def __init__(self, monkeypatch):
        self.device, self.stream, self.capturing, self.made = 0, "main", set(), []
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(torch.cuda, "device", lambda d: self.swap("device", d))
        monkeypatch.setattr(torch.cuda, "stream", lambda s: self.swap("stream", s))
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing",
                            lambda: self.stream in self.capturing)
        monkeypatch.setattr(tv.torch, "empty", self.empty)
        monkeypatch.setattr(tv, "_ws_cache", {})

    @contextlib.contextmanager
    def swap(self, what, value):
        old = getattr(self, what)
        if value is not None:
            setattr(self, what, value)
        yield
        setattr(self, what, old)

    def empty(self, n, dtype=None, device=None):
        self.made.append((n, self.device, self.stream, device))
        return torch.zeros(n, dtype=dtype)


@pytest.fixture
def cuda(monkeypatch):
    return FakeCuda(monkeypatch)


def test_size_is_the_tensors_device_s(cuda):
    sizes = {0: 100, 1: 200}
    ws = tv._scratch("prefill", 1, None, 7, lambda x: sizes[cuda.device] + x, 5)
    assert ws.numel() == 205 and cuda.made == [(205, 1, "main", "cuda:1")]
    assert cuda.device == 0


def test_allocated_on_the_stream_that_uses_it(cuda):
    tv._scratch("pages", 0, "side", 9, lambda x: x, 64)
    assert cuda.made == [(64, 0, "side", "cuda:0")] and cuda.stream == "main"


@pytest.mark.parametrize("given", [None, "graph"])
def test_a_capture_has_its_own(cuda, given):
    kept = tv._scratch("pages", 0, None, 9, lambda x: x, 64)
    assert tv._scratch("pages", 0, None, 9, lambda x: x, 32) is kept
    cuda.capturing = {"graph"}
    with cuda.swap("stream", "graph" if given is None else "main"):
        one = tv._scratch("pages", 0, given, 9, lambda x: x, 64)
        two = tv._scratch("pages", 0, given, 9, lambda x: x, 64)
    assert one is not two and one is not kept
    assert tv._scratch("pages", 0, None, 9, lambda x: x, 64) is kept


def test_nothing_needed_is_still_an_address(cuda):
    assert tv._scratch("prefill", 0, None, 9, lambda x: x, 0).numel() == 1
