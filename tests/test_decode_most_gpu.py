"""GPU tests of the rotations and norms with as many tokens, and sequences, as a call may name."""
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
T = 2 ** 31 - 1


@pytest.fixture
def many():
    """One pair a token, 8.6 GB, and every token's position."""
    x = torch.empty((T, 1, 2), dtype=torch.bfloat16, device="cuda")
    x.view(T, 2).copy_(torch.tensor([1.0, -0.5], device="cuda").bfloat16().expand(T, 2))
    yield x
    del x
    torch.cuda.empty_cache()


PARTS = [slice(first, first + 5000) for first in (0, 1 << 30, T - 5000)]


def test_rope_of_the_most_tokens(many):
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    want = [torch.empty_like(many[part]) for part in PARTS]
    for part, alone in zip(PARTS, want):
        tv.rope(many[part], alone, pos[part])
    tv.rope(many, many, pos)
    for part, alone in zip(PARTS, want):
        assert torch.equal(many[part], alone)


def test_norms_of_the_most_tokens(many):
    def i32(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    weight = torch.tensor([1.0, 2.0], device="cuda").bfloat16()
    out = torch.full_like(many, -77.0)
    tv.norm_rope(many, None, i32([0, T]), i32([0]), None, out, None, None, q_weight=weight)
    for part in PARTS:
        alone = torch.empty_like(many[part])
        tv.norm_rope(many[part], None, i32([0, 5000]), i32([part.start]), None, alone, None, None,
                     q_weight=weight)
        assert torch.equal(out[part], alone)


@pytest.mark.parametrize("B", [2 ** 31 - 1, 2 ** 31 - 32, 2 ** 30 + 5])
def test_norms_of_the_most_sequences(B):
    # all but three of them empty, ones before, between and behind
    i32 = dict(dtype=torch.int32, device="cuda")
    owner, n = [B // 3, B - 2, B - 1], [4, 1, 6]
    start, prefix = torch.zeros(B + 1, **i32), torch.zeros(B, **i32)
    at = 0
    for b, k in zip(owner, n):
        at += k
        start[b + 1:] = at
        prefix[b] = 100 + k
    g = torch.Generator(device="cuda").manual_seed(41)
    q = torch.randn((at + 2, 3, 64), generator=g, device="cuda").bfloat16()
    out, want = torch.full_like(q, -77.0), torch.full_like(q, -77.0)
    tv.norm_rope(q, None, start, prefix, None, out, None, None)
    tv.norm_rope(q, None, torch.tensor([0, 4, 5, 11], **i32), torch.tensor([104, 101, 106], **i32),
                 None, want, None, None)
    assert torch.equal(out, want) and (out[at:] == -77.0).all()
