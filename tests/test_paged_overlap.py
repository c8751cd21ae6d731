"""Outputs of the paged cache's calls that overlap their inputs are refused."""
from __future__ import annotations

import ctypes

import pytest
import torch

from kimi_delta_attention_32_b200 import kda
from test_paged_abi import INV, WS, _decode, _evict, lib      # noqa: F401

# Addresses that share nothing: q and o of [2, 8, 128] bf16 are 4096 bytes, a cache of 8 pages 65536
# each, and the workspace some megabytes.
AT = dict(q=1 << 30, z=2 << 30, o=3 << 30, kc=4 << 30, vc=5 << 30, bt=6 << 30, sl=7 << 30, acc=8 << 30,
          ws=9 << 30, pos=10 << 30, ao=11 << 30, qo=12 << 30, so=13 << 30)
DECODE, EVICT = ("q", "z", "o", "kc", "vc", "bt", "sl", "acc", "ws"), \
    ("kc", "vc", "bt", "sl", "acc", "pos", "ao", "qo", "so", "ws")


def _call(fn, names, lib, **kw):        # noqa: F811
    a = {n: AT[n] for n in names}
    a.update(slots=64, **kw)
    return fn(lib, **{k: ctypes.c_void_p(v) if k in AT else v for k, v in a.items()})


@pytest.mark.parametrize("other,by", [
    ("q", 0), ("q", 16), ("q", -16), ("q", 4080), ("z", 0), ("z", -4080), ("kc", 0), ("kc", 65536 - 16),
    ("vc", -16), ("vc", 32768), ("bt", -4080), ("sl", -4080), ("acc", 1008), ("ws", 0), ("ws", 4096)])
def test_decode_refuses_an_output_over_its_inputs(lib, other, by):       # noqa: F811
    assert _call(_decode, DECODE, lib, o=AT[other] + by) == INV
    assert _call(_decode, DECODE, lib, o=AT[other] + by, ws=0) == WS


def test_decode_refuses_an_output_in_pages_far_apart(lib):       # noqa: F811
    """Pages every megabyte: each page is looked at, the last one too."""
    for page in (0, 1, 7):
        for by in (-16, 0, 8176):
            assert _call(_decode, DECODE, lib, ps=1 << 19, o=AT["vc"] + (page << 20) + by) == INV


@pytest.mark.parametrize("kw", [dict(ao="pos"), dict(qo="acc"), dict(ao="qo"), dict(qo="ao")])
@pytest.mark.parametrize("by", [0, 512])
def test_evict_refuses_outputs_over_each_other(lib, kw, by):       # noqa: F811
    assert _call(_evict, EVICT, lib, **{k: AT[v] + by for k, v in kw.items()}) == INV


@pytest.mark.gpu
def test_outputs_beside_and_between_the_inputs_are_taken():
    """One allocation holds a page's rows, q, o and z in turn, page after page: nothing overlaps."""
    d, H, page, pages, N, Hq = 64, 2, 16, 4, 2, 4
    rows, qs = page * H * d, N * Hq * d
    room = torch.randn(pages, 2 * rows + 3 * qs, dtype=torch.float32).to(torch.bfloat16).to("cuda")

    def part(at, shape):
        return room[:, at:at + shape[-1] * shape[-2] * shape[-3]].unflatten(1, shape)
    k, v = part(0, (page, H, d)), part(rows, (page, H, d))
    q, o, z = (room[2, 2 * rows + i * qs:2 * rows + (i + 1) * qs].view(N, Hq, d) for i in range(3))
    table = torch.tensor([[0, 1], [3, 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 32], dtype=torch.int32, device="cuda")
    apart = [t.clone() for t in (q, k, v, z)]
    want = kda.paged_decode(*apart[:3], table, lens, scale=0.2, z=apart[3])
    kda.paged_decode(q, k, v, table, lens, scale=0.2, z=z, o=o)
    assert torch.equal(o, want)
    for t, s in zip((q, k, v, z), apart):
        assert torch.equal(t, s)
    with pytest.raises(kda.KdaError):
        kda.paged_decode(q, k, v, table, lens, scale=0.2, o=q)
    with pytest.raises(kda.KdaError):
        kda.paged_decode(q, k, v, table, lens, scale=0.2, z=z, o=z)
