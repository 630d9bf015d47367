"""GPU tests of tv_token_sample on bf16 rows whose values the table of weights cannot hold at once:
logits that cross zero, from ordinary magnitudes down to those next to it.  Equal to the rule in 64
bits, as in test_token_gpu.py."""
import numpy as np
import pytest
import torch

from tests import test_token_gpu as tokens

pytestmark = [pytest.mark.gpu, pytest.mark.usefixtures("tvlib")]
V = 120011         # eight CTAs a row, each with enough of it for the table
FILTERS = [dict(), dict(p=0.7), dict(p=0.95), dict(k=90000, p=0.7), dict(p=0.7, m=0.3)]


def check(x, seed, **kw):
    u = torch.rand(len(x), generator=torch.Generator().manual_seed(seed)).numpy()
    tokens.check(x.bfloat16(), u, **kw)


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("largest", [0.0, 1e-38, 1e-30, 1e-12, 3.0])
def test_logits_next_to_zero(kw, largest):
    # below the largest one: magnitudes of each size, and of all sizes
    g = torch.Generator().manual_seed(51)
    size = torch.tensor([1e-39, 1e-30, 1e-20, 1e-12, 1e-8, 1e-3, 1.0])[:, None]
    x = -torch.randn((8, V), generator=g).abs()
    x[:7] *= size
    x[7] *= torch.exp(-90 * torch.rand(V, generator=g))
    x[:, 7777] = largest
    check(x, 52, **kw)


@pytest.mark.parametrize("kw", FILTERS)
@pytest.mark.parametrize("temperature", [2e-30, 1e-20, 1e-6, 0.05])
def test_logits_of_the_temperature_and_below(kw, temperature):
    g = torch.Generator().manual_seed(53)
    x = torch.randn((8, V), generator=g) * temperature
    x[1::2] = -x[1::2].abs()
    x[2:4] *= torch.exp(-60 * torch.rand((2, V), generator=g))
    x[4:6] *= 1e-6
    check(x.clamp(-3e38, 3e38), 54, temperature=temperature, **kw)


@pytest.mark.parametrize("kw", FILTERS[:3])
def test_lightest_logits_next_to_zero(kw):
    # the weights' end, 60 log2 units below the maximum, lies next to zero on either side
    g = torch.Generator().manual_seed(55)
    x = torch.rand((8, V), generator=g) * 41.0
    x *= torch.where(torch.rand((8, V), generator=g) < 0.5, torch.tensor(1e-9), torch.tensor(1.0))
    x[4:] *= -1e-3
    x[:, 5] = torch.tensor([41.5, 41.75] * 4)
    check(x, 56, **kw)
