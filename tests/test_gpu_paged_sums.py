"""GPU tests of the sums of one-token attention over very long caches."""
from __future__ import annotations

import pytest
import torch

from kimi_delta_attention_32_b200 import kda
from test_gpu_paged import Paged, check_decode

pytestmark = pytest.mark.gpu
DEV = "cuda"


def values_with_mean(n, d, mean, seed):
    """bf16 [n, d] whose channels' exact means lie within 2^-6 / n of `mean`: large values in the even
    rows, small ones with many low bits in the odd rows."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(n, d, generator=g, dtype=torch.float64)
    v[0::2] = 2 * mean + v[0::2] / 4
    v[1::2] /= 64
    v = v.to(torch.bfloat16).double()
    steps = torch.round((n * mean - v.sum(0)) * 64)              # values in [2, 4) are 2^-6 apart
    room = (v > 2.1) & (v < 3.9)
    chosen = room & (room.cumsum(0) <= steps.abs())
    v += chosen * steps.sign() / 64
    assert torch.equal(v, v.to(torch.bfloat16).double())
    return v


@pytest.mark.parametrize("d", [64, 128])
def test_long_sums_do_not_drift(d):
    """Equal weights over 262144 values, by blocks that walk whole sequences. The exact means lie
    2^-15 above the middle of two bf16, so every output is the upper one unless the sums lose more
    than that. Each warp of four adds 4096 steps of 16 slots, whose sums are exact to 2^-24 of their
    largest value. Rounded to nearest, each addition errs by at most 2^-24 of the sum so far, up or
    down: sqrt(4096 / 3) / 2 of these together, at 8 standard deviations 2^-24 * 151 = 9e-6 < 2^-15.
    Additions that are cut instead all err downwards: about 0.72 * 2^-24 * 4096 / 2 = 9e-5."""
    n, page = 262144, 64
    mean = 1 + 2.0 ** -8 + 2.0 ** -15
    v = values_with_mean(n, d, mean, d)
    assert ((v.sum(0) / n - mean).abs() < 2.0 ** -20).all()
    vc = v.to(torch.bfloat16).view(n // page, page, 1, d).to(DEV)
    N = 3 * torch.cuda.get_device_properties(0).multi_processor_count      # a sequence a block at least
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).expand(N, -1).contiguous()
    lens = torch.full((N,), n, dtype=torch.int32, device=DEV)
    q = torch.zeros(N, 1, d, dtype=torch.bfloat16, device=DEV)
    o = kda.paged_decode(q, torch.zeros_like(vc), vc, table, lens)
    assert kda.last_device_error() == kda.KDA_OK
    assert torch.equal(o, torch.full_like(o, 1 + 2.0 ** -7)), o.double().mean().item()


@pytest.mark.parametrize("io,d,tile", [("bf16", 128, 64), ("bf16", 64, 64), ("f32", 64, 64), ("f32", 128, 128)])
@pytest.mark.parametrize("tiles", [2, 3, 4, 5, 6])
def test_outputs_do_not_depend_on_the_weights_being_gathered(io, d, tile, tiles):
    """On both sides of the length up to which a block takes a whole segment."""
    c = Paged(io, [tile * tiles, tile * tiles - 5, 1], 2, d, 16, seed=tiles)
    q = c.rand(3, 8, d)
    acc = c.acc.clone()
    o = kda.paged_decode(q, *c.args, scale=0.2, acc=acc, max_len=tile * tiles)
    check_decode(c, q, o, 0.2, None, acc, c.acc)
    assert torch.equal(o, kda.paged_decode(q, *c.args, scale=0.2, max_len=tile * tiles))
