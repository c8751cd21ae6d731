"""GPU tests of one-token attention with values at the ends of their type's range."""
from __future__ import annotations

import pytest
import torch

from kimi_delta_attention_32_b200 import kda
from test_gpu_paged import Paged, check_decode

pytestmark = pytest.mark.gpu


def near_the_top(like, seed):
    """fp32 values of both signs between (2 - 2^-10) 2^127 and the largest one, that among them; NaN
    stays where `like` has it."""
    g = torch.Generator().manual_seed(seed)
    bits = torch.randint(0x7f7fe000, 0x7f800000, like.shape, generator=g, dtype=torch.int32)
    bits.view(-1)[::5] = 0x7f7fffff
    x = bits.view(torch.float32) * torch.where(torch.rand(like.shape, generator=g) < 0.5, -1.0, 1.0)
    return torch.where(like.isnan(), like, x.to(like.device))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G", [1, 8, 12])
def test_largest_fp32_values(d, G):
    """One entry that takes all the weight: the output is its value, however large."""
    c = Paged("f32", [1, 1, 1], 2, d, 16, seed=G)
    c.v = near_the_top(c.v, d)
    q = c.rand(3, 2 * G, d)
    acc = c.acc.clone()
    o = kda.paged_decode(q, *c.args, scale=0.1, acc=acc)
    check_decode(c, q, o, 0.1, None, acc, c.acc)


@pytest.mark.parametrize("large", ["keys", "queries"])
def test_largest_fp32_operands_of_scores(large):
    """Keys or queries at the top of the range, the other side small: ordinary scores."""
    c = Paged("f32", [40, 130, 1], 2, 64, 16, seed=5)
    q = c.rand(3, 8, 64)
    if large == "keys":
        c.k, q = near_the_top(c.k, 1), q * 2.0 ** -100
    else:
        c.k, q = c.k * 2.0 ** -100, near_the_top(q, 1)
    acc = c.acc.clone()
    o = kda.paged_decode(q, *c.args, scale=2.0 ** -30, acc=acc)
    check_decode(c, q, o, 2.0 ** -30, None, acc, c.acc)
