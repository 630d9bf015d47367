"""GPU tests of the decode calls without tokens, sequences or rows: nothing is read or written."""
import pytest
import torch

from speculative_decoding_tree_04_gb300 import tv

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]


def bf16(*shape):
    return torch.full(shape, -77.0, dtype=torch.bfloat16, device="cuda")


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("q,kv", [(True, True), (True, False), (False, True)])
@pytest.mark.parametrize("B", [0, 3])
def test_norm_rope_without_tokens(q, kv, B):
    c, k = bf16(64, 512), bf16(64, 64)
    tv.norm_rope(bf16(0, 4, 96) if q else None, bf16(0, 576) if kv else None, i32([0] * (B + 1)),
                 i32([5] * B), bf16(0, 4, 32), bf16(0, 4, 64), c, k,
                 page_table=i32([[0, 1]] * B).view(B, 2))
    torch.cuda.synchronize()
    assert (c == -77.0).all() and (k == -77.0).all()


def test_rope_without_tokens():
    x = bf16(0, 4, 64)
    tv.rope(x, x, i32([]))
    tv.rope(x, bf16(0, 4, 64), i32([]))


def test_shared_attn_without_sequences():
    c, k = bf16(64, 512), bf16(64, 64)
    for start, shared in ((None, None), (i32([0]), i32([]))):
        tv.shared_attn(bf16(0, 1, 4, 512), bf16(0, 1, 4, 64), c, k, i32([]), start, shared,
                       bf16(0, 1, 4, 512), torch.empty((0, 1, 4), device="cuda"), 0.1,
                       max_prefix_len=0, page_table=i32([]).view(0, 2))


def test_token_sample_without_rows():
    none = torch.empty(0, device="cuda")
    tv.token_sample(bf16(0, 100), none, i32([]), temperature=none, top_k=i32([]), kept=i32([]))
