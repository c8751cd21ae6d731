"""GPU tests of the paged cache's calls on caches with bad pages, on very large ones, and with host
bounds far above the lengths."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import paged_ref as ref
from kimi_delta_attention_32_b200 import kda
from test_gpu_paged import DEV, Paged, check_decode, evict_case, f64

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


def loosened(c, slots):
    """The same cache with a table and side arrays for so many slots a sequence."""
    wide = torch.full((len(c.lens), -(-slots // c.page)), -1, dtype=torch.int32)
    wide[:, :c.max_pages] = c.table
    c.table, c.tab, c.max_pages = wide, wide.to(DEV), wide.shape[1]
    more = slots - c.slots
    c.acc = torch.nn.functional.pad(c.acc, (0, more), value=0.5)
    c.pos = torch.nn.functional.pad(c.pos, (0, more), value=7)
    c.slots = slots
    return c


@pytest.mark.parametrize("slots", [1500, 9000, 70000, 400000, 1 << 20])
def test_evict_with_a_bound_far_above_the_lengths(slots):
    """Blocks, threads and shared memory follow the bound, the keys that a block holds its part of a
    sequence."""
    for in_place in (False, True):
        c = loosened(Paged("bf16", [1200, 300, 65, 41, 0], 2, 64, 16, seed=slots), slots)
        evict_case(c, 40, 2, 6, in_place=in_place)
        c = loosened(Paged("f32", [1200, 300], 1, 64, 7, seed=slots), slots)
        evict_case(c, 700, 2, 6, in_place=in_place)


def test_evict_short_sequences_beside_one_too_long_for_shared_memory():
    for in_place in (False, True):
        c = Paged("bf16", [400100, 9000, 300, 10], 1, 64, 128, seed=3)
        evict_case(c, 8000, 16, 1000, in_place=in_place)


@pytest.mark.parametrize("io,H,G", [("bf16", 2, 4), ("f32", 1, 12)])
@pytest.mark.parametrize("slots", [1500, 70000, 1 << 20])
def test_decode_with_a_bound_far_above_the_lengths(io, H, G, slots):
    c = loosened(Paged(io, [1200, 300, 65, 0, 1], H, 64, 16, seed=slots), slots)
    q, acc = c.rand(5, H * G, 64), c.acc.clone()
    o = kda.paged_decode(q, *c.args, scale=0.2, acc=acc)
    assert kda.last_device_error() == kda.KDA_OK
    check_decode(c, q, o, 0.2, None, acc, c.acc)


def test_evict_offsets_beyond_32_bits():
    """Keys and values of a cache of more than 2^31 elements."""
    H, d, page = 8, 128, 64
    P = 2 ** 31 // (H * d * page) + 40
    k = torch.empty(P, page, H, d, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    c = Paged("bf16", [500, 260], H, d, page, seed=7)
    first = P - c.k.shape[0]
    k[first:], v[first:] = c.k, c.v
    K, V, A, Q = (f64(t) for t in (c.k, c.v, c.acc, c.pos))
    want = ref.evict(K, V, c.table.numpy(), c.lens, 200, A, Q, c.lens, 2, 30)
    out = kda.cache_evict(k, v, torch.where(c.tab >= 0, c.tab + first, c.tab), c.sl, 200, c.acc, c.pos,
                          n_first=2, n_recent=30)
    assert kda.last_device_error() == kda.KDA_OK and out.tolist() == want
    assert np.array_equal(f64(k[first:]), K, equal_nan=True)
    assert np.array_equal(f64(v[first:]), V, equal_nan=True)
    assert np.array_equal(f64(c.acc)[:, :, :200], A[:, :, :200])
    assert np.array_equal(f64(c.pos)[:, :, :200], Q[:, :, :200])
