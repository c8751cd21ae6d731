"""GPU tests of the paged cache's eviction on caches with bad pages, and on very large ones."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_ref as ref
from kimi_delta_attention_32_b200 import kda
from test_gpu_paged import DEV, Paged, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,d,page", [("bf16", 64, 16), ("f32", 128, 7), ("bf16", 128, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_rows_of_bad_pages_are_zeros(io, d, page, in_place):
    """A free slot that an entry on a bad page fills keeps nothing of the entry before: key and value
    are zeros, weight and position the new entry's. Rows that would move to a bad page are dropped."""
    lens, keep = [200, 160, 30], 50
    c = Paged(io, lens, 2, d, page, seed=page)
    P = c.k.shape[0]
    for n, slots in ((0, (3, 49, 70, 100, 185, 199)), (1, (0, 90, 150))):
        for s in slots:
            c.table[n, s // page] = (-1, P, 1 << 30)[s % 3]
    c.tab = c.table.to(DEV)
    t = c.table.numpy().copy()                           # for the reference: pages of their own, of zeros
    bad = np.argwhere((t < 0) | (t >= P))
    bad = [(n, e) for n, e in bad if e * page < lens[n]]
    K, V = (np.concatenate([f64(x), np.zeros((len(bad), page, 2, d))]) for x in (c.k, c.v))
    for i, (n, e) in enumerate(bad):
        t[n, e] = P + i
    A, Q = f64(c.acc), f64(c.pos)
    want = ref.evict(K, V, t, lens, keep, A, Q, lens, 4, 20)
    ao, po = (c.acc, c.pos) if in_place else (torch.zeros_like(c.acc), torch.zeros_like(c.pos))
    out = kda.cache_evict(*c.args, keep, c.acc, c.pos, n_first=4, n_recent=20, acc_out=ao, pos_out=po)
    assert kda.last_device_error() == kda.KDA_ERR_INDEX
    assert out.tolist() == want
    assert np.array_equal(f64(c.k), K[:P], equal_nan=True)
    assert np.array_equal(f64(c.v), V[:P], equal_nan=True)
    assert (K[:P] == 0).all(-1).any()                    # the case occurs
    for n, m in enumerate(want):
        assert np.array_equal(f64(ao)[n, :, :m], A[n, :, :m])
        assert np.array_equal(f64(po)[n, :, :m], Q[n, :, :m])
