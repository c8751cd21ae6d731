"""GPU tests of the paged key-value cache's operators against their fp64 forms (paged_ref)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import paged_ref as ref
from kimi_delta_attention_32_b200 import kda

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
DEV = "cuda"


def f64(t):
    return t.detach().cpu().double().numpy()


class Paged:
    """A cache of random rows with shuffled pages; rows that no sequence holds are NaN."""

    def __init__(self, io, lens, H, d, page, layout="token", seed=0, room=0, extra_pages=2, acc=True):
        self.io, self.H, self.d, self.page, self.lens = io, H, d, page, list(lens)
        g = torch.Generator().manual_seed(seed)
        self.g = g
        N = len(lens)
        need = [-(-(n + room) // page) for n in lens]
        P = sum(need) + extra_pages
        perm = torch.randperm(P, generator=g)
        self.max_pages = max(1, max(need, default=1))
        table = torch.full((N, self.max_pages), -1, dtype=torch.int32)
        at = 0
        for n, k in enumerate(need):
            table[n, :k] = perm[at:at + k].int()
            at += k
        live = torch.zeros(P, page, dtype=torch.bool)
        for n, length in enumerate(lens):
            p, r = ref.place(table.numpy(), n, np.arange(length), page)
            live[p, r] = True
        self.table = table
        self.slots = max(1, max(n + room for n in lens) if lens else 1)

        def pages():
            x = torch.randn(P, page, H, d, generator=g).to(DT[io])
            x[~live] = float("nan")
            x = x.to(DEV)
            if layout == "head":
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            return x
        if layout == "pair":                       # K and V interleaved page by page
            kv = torch.empty(P, 2, page, H, d, dtype=DT[io], device=DEV)
            kv[:, 0], kv[:, 1] = pages(), pages()
            self.k, self.v = kv[:, 0], kv[:, 1]
        elif layout == "padded":                   # rows with a gap behind them
            k, v = (torch.full((P, page, H, d + 8), float("nan"), dtype=DT[io], device=DEV)
                    for _ in range(2))
            k[..., :d], v[..., :d] = pages(), pages()
            self.k, self.v = k[..., :d], v[..., :d]
        else:
            self.k, self.v = pages(), pages()
        self.tab = table.to(DEV)
        self.sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.acc = torch.rand(N, H, self.slots, generator=g).to(DEV)
        self.pos = torch.arange(self.slots, dtype=torch.int32).expand(N, H, -1).contiguous().to(DEV)

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g).to(DT[self.io]).to(DEV)

    @property
    def args(self):
        return self.k, self.v, self.tab, self.sl


def check_decode(c, q, o, scale, z=None, acc=None, acc0=None, skip=None, lens=None):
    lens = c.lens if lens is None else lens
    r, weights, mag, rel = ref.decode(f64(q), f64(c.k), f64(c.v), c.table.numpy(), lens, scale,
                                      None if z is None else f64(z), skip)
    bound = ref.decode_bound(c.io, r, mag, rel)
    err = np.abs(f64(o) - r)
    assert np.all(np.isfinite(f64(o)))
    assert np.all(err <= bound), f"o: {np.max(err / bound):.3g} of its bound"
    if acc is None:
        return
    got, old = f64(acc), f64(acc0)
    G = q.shape[1] // c.H
    for n, w in enumerate(weights):
        length = lens[n]
        rb = rel[n].reshape(c.H, G).max(1)[:, None]
        want = old[n, :, :length] + w
        assert np.all(np.abs(got[n, :, :length] - want) <= rb * w + 2 * ref.U24 * np.abs(want) + 1e-30)
        assert np.array_equal(got[n, :, length:], old[n, :, length:])      # slots behind the end


def decode_case(io, lens, Hq, H, d, page, layout="token", gate=False, acc=False, seed=0, scale=None):
    c = Paged(io, lens, H, d, page, layout, seed)
    q, z = c.rand(len(lens), Hq, d), c.rand(len(lens), Hq, d) if gate else None
    scale = d ** -0.5 if scale is None else scale
    a = c.acc.clone() if acc else None
    o = kda.paged_decode(q, *c.args, scale=scale, z=z, acc=a)
    torch.cuda.synchronize()
    assert kda.last_device_error() == kda.KDA_OK
    check_decode(c, q, o, scale, z, a, c.acc)
    return c, q, o


# lengths around the 16-slot and 64-slot steps of a tile, empty and single ones among them
EDGE = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("G,H", [(1, 3), (4, 2), (8, 2), (12, 1), (32, 1)])
@pytest.mark.parametrize("more", [[], [1500]], ids=["whole", "divided"])
def test_decode_edge_lengths(io, d, G, H, more):
    """The short ones alone are a block each; with a long one among them the tiles are divided."""
    decode_case(io, EDGE + more, G * H, H, d, 16, gate=True, acc=True, seed=G)


@pytest.mark.parametrize("lens,Hq,H", [([2000, 100], 71, 1), ([700, 0, 1300], 48, 2), ([1100] * 5, 20, 1)])
def test_decode_divided_groups(lens, Hq, H):
    """Groups of several head tiles, whose segments the division cuts."""
    decode_case("bf16", lens, Hq, H, 128, 24, gate=True, acc=True, seed=Hq)
    decode_case("f32", lens, Hq, H, 64, 32, acc=True, seed=Hq)


@pytest.mark.parametrize("G", [2, 3, 5, 7, 9, 16, 17, 24, 33, 71])
def test_decode_group_sizes(G):
    decode_case("bf16", [70, 3, 300], 2 * G, 2, 128, 32, acc=True, seed=G)
    decode_case("f32", [70, 3], G, 1, 64, 32, acc=True, seed=G)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 24, 48, 64, 100, 257, 1024])
@pytest.mark.parametrize("layout", ["token", "head", "pair", "padded"])
def test_decode_pages_and_strides(page, layout):
    decode_case("bf16", [333, 0, 64, 1], 8, 2, 128, page, layout, acc=True, seed=page)
    decode_case("f32", [130, 5], 8, 2, 64, page, layout, seed=page)


@pytest.mark.parametrize("io,N,L,Hq,H", [("bf16", 1, 20000, 8, 1), ("bf16", 2, 9001, 32, 4),
                                         ("f32", 1, 20001, 4, 1), ("bf16", 3, 5000, 40, 1)])
def test_decode_long(io, N, L, Hq, H):
    """Few rows over a long cache: the length is split and the parts joined."""
    decode_case(io, [L - 7 * n for n in range(N)], Hq, H, 128, 64, gate=True, acc=True, seed=L)


def test_decode_many_sequences():
    g = np.random.default_rng(5)
    decode_case("bf16", [int(x) for x in g.integers(0, 40, 700)], 4, 2, 64, 16, acc=True, seed=1)


@pytest.mark.parametrize("N", [31, 32, 33, 64, 65, 1100, 5000])
def test_decode_batch_sizes(N):
    """Around the 32 sequences that a warp scans at once, and many of them, empty runs among them."""
    g = np.random.default_rng(N)
    lens = [0 if 10 <= i < 50 and N > 64 else int(x) for i, x in enumerate(g.integers(0, 70, N))]
    decode_case("f32", lens, 2, 1, 64, 16, acc=True, seed=N)


def test_decode_only_empty_sequences():
    c = Paged("bf16", [0, 0, 0], 2, 128, 16)
    q = c.rand(3, 4, 128)
    acc = c.acc.clone()
    o = kda.paged_decode(q, *c.args, z=q, acc=acc, max_len=0, o=torch.full_like(q, 7.0))
    assert torch.count_nonzero(o) == 0 and torch.equal(acc, c.acc)
    assert kda.last_device_error() == kda.KDA_OK


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decode_large_scores(io):
    """Scores of several hundred: the running maximum keeps the exponentials in range, and one
    entry takes all the weight."""
    c = Paged(io, [500, 40], 2, 64, 16, seed=3)
    q = c.rand(2, 4, 64) * 8
    o = kda.paged_decode(q, *c.args, scale=4.0)
    assert torch.isfinite(o).all()
    x = torch.einsum("nhgd,nhsd->nhgs", q.view(2, 2, 2, 64).double(), torch.stack(
        [c.k[c.tab[n].clamp(min=0).long()].reshape(-1, 2, 64)[:40].transpose(0, 1) for n in range(2)]
    ).double()) * 4.0
    assert x.abs().max() > 300
    # scores this large leave their fp32 rounding in the weights: the bound follows from it
    check_decode(c, q, o, 4.0)


def test_decode_equal_scores_average():
    c = Paged("f32", [77], 1, 64, 16)
    q = torch.zeros(1, 2, 64, device=DEV)
    acc = torch.zeros_like(c.acc)
    o = kda.paged_decode(q, *c.args, acc=acc)
    check_decode(c, q, o, 1.0, None, acc, torch.zeros_like(acc))


def test_decode_skips_bad_pages_and_clamps_lengths():
    """Page numbers out of range are left out, lengths out of range clamped; both are reported once."""
    for io in ("f32", "bf16"):
        c = Paged(io, [100, 64, 30, 50], 2, 64, 16, seed=4)
        c.table[0, 2], c.table[0, 5], c.table[1, :4] = -1, c.k.shape[0], 1 << 30
        c.tab = c.table.to(DEV)
        q = c.rand(4, 8, 64)
        acc = c.acc.clone()
        o = kda.paged_decode(q, *c.args, acc=acc)
        assert kda.last_device_error() == kda.KDA_ERR_INDEX
        assert kda.last_device_error() == kda.KDA_OK
        check_decode(c, q, o, 1.0, None, acc, c.acc,
                     skip=lambda p: (p < 0) | (p >= c.k.shape[0]))
        assert torch.count_nonzero(o[1]) == 0                       # nothing left to attend to
        c = Paged(io, [100, 64, 30, 50], 2, 64, 16, seed=4)
        c.sl[2], c.sl[3] = -5, 51                                   # max_len 50 below
        o = kda.paged_decode(q, *c.args, max_len=50)
        assert kda.last_device_error() == kda.KDA_ERR_INDEX
        check_decode(c, q, o, 1.0, lens=[50, 50, 0, 50])


def test_decode_offsets_beyond_32_bits():
    """A cache of more than 2^31 elements; the sequences' pages lie at its end."""
    H, d, page = 8, 128, 64
    P = 2 ** 31 // (H * d * page) + 40
    k = torch.empty(P, page, H, d, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    c = Paged("bf16", [500, 260], H, d, page, seed=6)
    first = P - c.k.shape[0]
    k[first:], v[first:] = c.k, c.v
    q = c.rand(2, 32, d)
    acc = c.acc.clone()
    o = kda.paged_decode(q, k, v, torch.where(c.tab >= 0, c.tab + first, c.tab), c.sl, scale=0.1,
                         acc=acc)
    check_decode(c, q, o, 0.1, None, acc, c.acc)
    # the same pages for the writes
    tab = torch.where(c.tab >= 0, c.tab + first, c.tab)
    new = c.rand(2, 1, H, d)
    kda.cache_append(new, -new, k, v, tab, c.sl - 1)
    for n, length in enumerate(c.lens):
        p, r = int(tab[n, (length - 1) // page]), (length - 1) % page
        assert torch.equal(k[p, r], new[n, 0]) and torch.equal(v[p, r], -new[n, 0])
    a0, p0, k0 = c.acc.clone(), c.pos.clone(), k[first:].clone()
    out = kda.cache_evict(k, v, tab, c.sl, 200, c.acc, c.pos)
    assert out.tolist() == [200, 200]
    K, V, A, Q = f64(k0), f64(k0), f64(a0), f64(p0)
    ref.evict(K, V, c.table.numpy(), c.lens, 200, A, Q, c.lens, 0, 0)
    assert np.array_equal(f64(k[first:]), K, equal_nan=True)


def test_decode_is_deterministic_and_leaves_its_inputs():
    c = Paged("bf16", [3000, 10, 700], 2, 128, 16, seed=8)
    q, z = c.rand(3, 16, 128), c.rand(3, 16, 128)
    saved = [t.clone() for t in (q, z, c.k, c.v, c.tab, c.sl)]
    runs = []
    for _ in range(3):
        acc = c.acc.clone()
        runs.append((kda.paged_decode(q, *c.args, z=z, acc=acc, scale=0.1), acc))
    for o, a in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(a, runs[0][1])
    for t, s in zip((q, z, c.k, c.v, c.tab, c.sl), saved):
        assert torch.equal(t.view(torch.uint8) if t.is_contiguous() else t.contiguous().view(torch.uint8),
                           s.contiguous().view(torch.uint8))


def test_decode_without_gate_or_weights_matches_with():
    c = Paged("bf16", [1000, 33], 2, 128, 16, seed=9)
    q = c.rand(2, 8, 128)
    o = kda.paged_decode(q, *c.args, scale=0.1)
    assert torch.equal(o, kda.paged_decode(q, *c.args, scale=0.1, acc=c.acc.clone()))
    assert torch.equal(o, kda.paged_decode(q, *c.args, scale=0.1, z=torch.full_like(q, 100.0)))


def test_decode_ignores_workspace_contents():
    c = Paged("bf16", [5000, 0, 33], 1, 128, 16, seed=10)
    q = c.rand(3, 4, 128)
    size = kda.paged_decode_workspace_size(3, 4, 1, 128, c.max_pages * 16, with_acc=True)
    outs = []
    for fill in (0, 255):                       # zeros; NaN and -1 everywhere
        ws = torch.full((size,), fill, dtype=torch.uint8, device=DEV)
        acc = torch.zeros(3, 1, c.max_pages * 16, device=DEV)
        outs.append((kda.paged_decode(q, *c.args, acc=acc, workspace=ws), acc))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_decode_stays_inside_its_workspace():
    c = Paged("bf16", [5000, 100, 700], 2, 128, 16, seed=11)
    q = c.rand(3, 80, 128)
    for acc in (None, c.acc):
        size = kda.paged_decode_workspace_size(3, 80, 2, 128, 5000, with_acc=acc is not None)
        ws = torch.full((size + 4096,), 77, dtype=torch.uint8, device=DEV)
        kda.paged_decode(q, *c.args, acc=acc, max_len=5000, workspace=ws[:size])
        assert (ws[size:] == 77).all()


def test_two_streams_at_once():
    """Two calls that overlap, each on its own stream and workspace."""
    cs = [Paged("bf16", [4000 + 500 * i, 90], 2, 128, 16, seed=20 + i) for i in range(2)]
    qs = [c.rand(2, 8, 128) for c in cs]
    want = [kda.paged_decode(q, *c.args, scale=0.1) for c, q in zip(cs, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    wss = [torch.empty(kda.paged_decode_workspace_size(2, 8, 2, 128, c.max_pages * 16),
                       dtype=torch.uint8, device=DEV) for c in cs]
    outs = [torch.empty_like(q) for q in qs]
    for _ in range(10):
        for c, q, s, ws, o in zip(cs, qs, streams, wss, outs):
            kda.paged_decode(q, *c.args, scale=0.1, workspace=ws, o=o, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert torch.equal(a, b)


def test_default_workspace_on_another_stream():
    """What a call allocates on its own belongs to the call's stream: work on the current stream,
    which soon takes over the freed memory, does not write into it."""
    c = Paged("bf16", [9000, 4000], 2, 128, 16, seed=21)
    q = c.rand(2, 8, 128)
    want = kda.paged_decode(q, *c.args, scale=0.1)
    size = kda.paged_decode_workspace_size(2, 8, 2, 128, c.max_pages * 16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for i in range(20):
        outs.append(kda.paged_decode(q, *c.args, scale=0.1, stream=s if i % 2 else s.cuda_stream))
        torch.full((size,), 255, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


def test_two_graphs_share_a_workspace():
    """Two captured calls with one workspace, replayed in turns."""
    cs = [Paged("bf16", [3000, 70], 2, 128, 16, seed=30), Paged("bf16", [500, 2000], 2, 128, 16, seed=31)]
    qs = [c.rand(2, 8, 128) for c in cs]
    want = [kda.paged_decode(q, *c.args, scale=0.1) for c, q in zip(cs, qs)]
    slots = max(c.max_pages for c in cs) * 16
    ws = torch.empty(kda.paged_decode_workspace_size(2, 8, 2, 128, slots), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros_like(q) for q in qs]
    graphs = []
    for c, q, o in zip(cs, qs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.paged_decode(q, *c.args, scale=0.1, workspace=ws, o=o)
        graphs.append(g)
    for _ in range(5):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            assert torch.equal(o, w)


def test_keys_that_are_the_values():
    """One tensor as both caches, and shared pages: reading needs no page to be a sequence's own."""
    c = Paged("bf16", [100, 100, 40], 2, 64, 16, seed=32)
    c.v = c.k
    c.table[1] = c.table[0]
    c.table[2, :3] = c.table[0, :3]
    c.tab = c.table.to(DEV)
    q = c.rand(3, 4, 64)
    acc = c.acc.clone()
    check_decode(c, q, kda.paged_decode(q, *c.args, scale=0.2, acc=acc), 0.2, None, acc, c.acc)


# ---------------------------------------------------------------- append

@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout,page", [("token", 16), ("head", 7), ("pair", 64), ("padded", 1)])
def test_append_packed(io, layout, page):
    lens, new = [0, 5, 16, 33, 7], [1, 0, 40, 3, 9]
    d, H = 64 if page == 7 else 128, 3
    c = Paged(io, lens, H, d, page, layout, room=40, seed=page)
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    k, v = c.rand(cu[-1], H, d), c.rand(cu[-1], H, d)
    seen = [x + 3 for x in lens]
    K, V, A, P = f64(c.k), f64(c.v), f64(c.acc), f64(c.pos)
    ref.append(K, V, c.table.numpy(), lens, f64(k), f64(v), cu, seen, A, P)
    sl = c.sl.clone()
    kda.cache_append(k, v, *c.args, positions=torch.tensor(seen, dtype=torch.int32, device=DEV),
                     acc=c.acc, pos=c.pos, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV),
                     cu_host=cu)
    assert kda.last_device_error() == kda.KDA_OK
    for t, r in ((c.k, K), (c.v, V), (c.acc, A), (c.pos, P)):
        assert np.array_equal(f64(t), r, equal_nan=True)
    assert torch.equal(c.sl, sl)


@pytest.mark.parametrize("T", [0, 1, 3])
def test_append_padded(T):
    lens = [0, 15, 16, 31]
    c = Paged("bf16", lens, 2, 128, 16, room=8)
    k, v = c.rand(4, T, 2, 128), c.rand(4, T, 2, 128)
    K, V, A, P = f64(c.k), f64(c.v), f64(c.acc), f64(c.pos)
    ref.append(K, V, c.table.numpy(), lens, f64(k).reshape(-1, 2, 128), f64(v).reshape(-1, 2, 128),
               [T * i for i in range(5)], None, A, P)
    kda.cache_append(k, v, *c.args, acc=c.acc, pos=c.pos)
    for t, r in ((c.k, K), (c.v, V), (c.acc, A), (c.pos, P)):
        assert np.array_equal(f64(t), r, equal_nan=True)
    kda.cache_append(k, v, *c.args)                     # without the side arrays
    kda.cache_append(k, v, *c.args, pos=c.pos)
    for t, r in ((c.k, K), (c.v, V), (c.acc, A), (c.pos, P)):
        assert np.array_equal(f64(t), r, equal_nan=True)


def test_append_drops_what_has_no_room():
    c = Paged("bf16", [14, 30, 3, 3], 2, 64, 16, room=2)
    c.sl = torch.tensor([14, 30, -2, 3], dtype=torch.int32, device=DEV)
    c.table[3, 0] = c.k.shape[0] + 5
    c.tab = c.table.to(DEV)
    k = c.rand(4, 4, 2, 64)
    before = f64(c.k)
    kda.cache_append(k, k, *c.args)
    assert kda.last_device_error() == kda.KDA_ERR_INDEX
    after = f64(c.k)
    # sequence 0 has room in its second table entry only if that names a page: -1 does not
    p, r = ref.place(c.table.numpy(), 0, [14, 15], 16)
    before[p, r] = f64(k)[0, :2]
    p, r = ref.place(c.table.numpy(), 1, [30, 31], 16)
    before[p, r] = f64(k)[1, :2]
    assert np.array_equal(before, after, equal_nan=True)
    acc = torch.ones(4, 2, 16, device=DEV)              # room for 16 slots only
    kda.cache_append(k, k, c.k, c.v, c.tab, torch.tensor([15, 16, 40, 0], dtype=torch.int32,
                                                         device=DEV), acc=acc)
    assert kda.last_device_error() == kda.KDA_ERR_INDEX
    want = torch.ones(4, 2, 16)
    want[0, :, 15] = 0
    assert torch.equal(acc.cpu(), want)


# ---------------------------------------------------------------- evict

def evict_case(c, keep, first=0, recent=0, seen=None, in_place=False, max_len=None):
    seen = c.lens if seen is None else seen
    K, V, A, P = (f64(t) for t in (c.k, c.v, c.acc, c.pos))
    A32 = c.acc.cpu().numpy().copy()
    want = ref.evict(K, V, c.table.numpy(), c.lens, keep, A, P, seen, first, recent)
    ao = c.acc if in_place else torch.full_like(c.acc, -3.0)
    po = c.pos if in_place else torch.full_like(c.pos, -3)
    so = c.sl if in_place else None
    s0 = c.sl.clone()
    out = kda.cache_evict(*c.args, keep, c.acc, c.pos, n_first=first, n_recent=recent,
                          positions=torch.tensor(seen, dtype=torch.int32, device=DEV),
                          acc_out=ao, pos_out=po, seqlens_out=so, max_len=max_len)
    assert kda.last_device_error() == kda.KDA_OK
    assert out.tolist() == want
    if not in_place:
        assert torch.equal(c.sl, s0)
        assert np.array_equal(c.acc.cpu().numpy(), A32, equal_nan=True)
    assert np.array_equal(f64(c.k), K, equal_nan=True) and np.array_equal(f64(c.v), V, equal_nan=True)
    for n, m in enumerate(want):
        assert np.array_equal(f64(ao)[n, :, :m], A[n, :, :m], equal_nan=True)
        assert np.array_equal(f64(po)[n, :, :m], P[n, :, :m])
        if not in_place:
            assert (ao[n, :, m:] == -3).all() and (po[n, :, m:] == -3).all()
    return want


@pytest.mark.parametrize("io,layout,page,d,H", [("bf16", "token", 16, 128, 2), ("f32", "head", 7, 64, 3),
                                                ("bf16", "pair", 64, 64, 1), ("f32", "padded", 1, 128, 2)])
@pytest.mark.parametrize("keep,first,recent", [(40, 4, 10), (64, 0, 0), (1, 0, 1), (0, 0, 0), (500, 3, 5)])
def test_evict(io, layout, page, d, H, keep, first, recent):
    for in_place in (False, True):
        c = Paged(io, [0, 1, 40, 41, 64, 65, 130, 300], H, d, page, layout, seed=keep)
        evict_case(c, keep, first, recent, in_place=in_place)


@pytest.mark.parametrize("kind", ["equal", "zeros", "two", "special", "negative"])
def test_evict_ties_and_special_weights(kind):
    c = Paged("bf16", [100, 257, 33], 2, 64, 16, seed=2)
    a = c.acc.cpu()
    if kind == "equal":
        a.fill_(0.25)
    elif kind == "zeros":                               # -0 and 0 are equal
        a = torch.where(torch.rand(a.shape) < 0.5, torch.zeros_like(a), -torch.zeros_like(a))
    elif kind == "two":
        a = (a > 0.6).float()
    elif kind == "special":
        for i, x in enumerate([float("nan"), float("inf"), -float("inf"), -float("nan"), 1e-45, 3e38]):
            a[..., i::11] = x
    else:
        a = -a
    c.acc = a.to(DEV)
    evict_case(c, 30, 2, 6)


@pytest.mark.parametrize("length,keep", [(131, 100), (9001, 5000), (9001, 9000), (30002, 128), (30003, 16384)])
@pytest.mark.parametrize("kind", ["nan", "steps", "runs"])
def test_evict_threshold_among_equals(length, keep, kind):
    """The keep-th best has equals in every warp's and block's slots; NaN is the lowest key of all,
    and the lengths end inside a group of four slots."""
    c = Paged("bf16", [length, length - 1, keep + 1], 1, 64, 16, seed=length + keep)
    a = c.acc.cpu()
    if kind == "nan":                                   # NaN entries have to stay
        a[torch.rand(a.shape, generator=c.g) < 0.995] = float("nan")
    elif kind == "steps":
        a = (a * 4).floor()
    else:
        a = torch.arange(c.slots).div(200, rounding_mode="floor").remainder(3).float().expand_as(a)
    c.acc = a.contiguous().to(DEV)
    evict_case(c, keep, 3, 20)


@pytest.mark.parametrize("off", [(0, 1, 2, 3), (1, 1, 1, 1), (4, 0, 4, 0), (0, 0, 0, 2)])
@pytest.mark.parametrize("slots", [5000, 5002])
def test_evict_alignment(off, slots):
    """acc, pos and their outputs at any multiple of 4 bytes."""
    c = Paged("bf16", [slots, 4100, 777], 3, 64, 16, seed=slots)
    K, V, A, P = (f64(t) for t in (c.k, c.v, c.acc, c.pos))
    want = ref.evict(K, V, c.table.numpy(), c.lens, 4001, A, P, c.lens, 4, 64)

    def at(x, by):
        room = torch.full((x.numel() + 8,), -3, dtype=x.dtype, device=DEV)
        view = room[by:by + x.numel()].view(x.shape)
        return room, view
    (_, a), (_, p), (ra, ao), (rp, po) = (at(x, by) for x, by in zip((c.acc, c.pos, c.acc, c.pos), off))
    a.copy_(c.acc)
    p.copy_(c.pos)
    out = kda.cache_evict(*c.args, 4001, a, p, n_first=4, n_recent=64, acc_out=ao, pos_out=po)
    assert kda.last_device_error() == kda.KDA_OK and out.tolist() == want
    assert np.array_equal(f64(c.k), K, equal_nan=True) and np.array_equal(f64(c.v), V, equal_nan=True)
    for n, m in enumerate(want):
        assert np.array_equal(f64(ao)[n, :, :m], A[n, :, :m])
        assert np.array_equal(f64(po)[n, :, :m], P[n, :, :m])
        assert (ao[n, :, m:] == -3).all() and (po[n, :, m:] == -3).all()
    for room, by in ((ra, off[2]), (rp, off[3])):
        assert (room[:by] == -3).all() and (room[by + c.acc.numel():] == -3).all()


@pytest.mark.parametrize("longest,keep", [(12001, 5000), (20003, 16000), (40000, 10001)])
def test_evict_more_heads_than_sms(longest, keep):
    """Blocks then hold more slots each: 1, 2 and 4 blocks a head."""
    g = np.random.default_rng(longest)
    lens = [longest] + [int(x) for x in g.integers(0, 400, 78)] + [longest - 1]
    c = Paged("bf16", lens, 2, 64, 16, seed=keep)
    evict_case(c, keep, 5, 100)


def test_evict_positions():
    """Guards go by position, not by slot: shuffled positions with gaps."""
    c = Paged("f32", [200, 90], 2, 64, 16, seed=12)
    g = torch.Generator().manual_seed(1)
    pos = torch.stack([torch.stack([torch.randperm(400, generator=g)[:c.slots] for _ in range(2)])
                       for _ in range(2)])
    c.pos = pos.int().to(DEV)
    evict_case(c, 60, 10, 20, seen=[400, 300])


@pytest.mark.parametrize("length,keep", [(5000, 4096), (4097, 4096), (70000, 30000), (70000, 69990),
                                         (70000, 3), (1025, 1000), (2048, 700), (2049, 700),
                                         (8193, 4000), (17000, 9000), (262145, 100000),
                                         (390000, 200000)])
def test_evict_long(length, keep):
    c = Paged("bf16", [length, length // 2, 10], 1, 64, 64, seed=length)
    evict_case(c, keep, 2 if keep > 3 else 0, keep // 4)


def test_evict_longer_than_the_keys_in_shared_memory():
    """More slots than one cluster's shared memory holds keys for."""
    length, keep = 500001, 400000
    c = Paged("bf16", [length], 1, 64, 128, seed=1)
    evict_case(c, keep, 16, 1000)


def test_evict_many_sequences():
    g = np.random.default_rng(2)
    c = Paged("bf16", [int(x) for x in g.integers(0, 60, 500)], 3, 64, 16, seed=5)
    evict_case(c, 25, 2, 5, in_place=True)


def test_evict_reports_bad_pages_and_lengths():
    c = Paged("bf16", [100, 60], 2, 64, 16, seed=13)
    c.table[0, 1] = -1
    c.tab = c.table.to(DEV)
    before = c.k.clone()
    a, p = c.acc.clone(), c.pos.clone()
    out = kda.cache_evict(*c.args, 20, a, p)
    assert kda.last_device_error() == kda.KDA_ERR_INDEX and out.tolist() == [20, 20]
    # the rows of the pages that exist moved as they should
    K, V, A, P = f64(before), f64(before), f64(c.acc), f64(c.pos)
    t = c.table.numpy().copy()
    t[0, 1] = c.k.shape[0]                               # a page of its own for the reference
    K = np.concatenate([K, K[:1]])
    ref.evict(K, K.copy(), t, c.lens, 20, A, P, c.lens, 0, 0)
    p1, r1 = ref.place(t, 1, np.arange(20), 16)
    assert np.array_equal(f64(c.k)[p1, r1], K[p1, r1])
    assert np.array_equal(f64(a)[:, :, :20], A[:, :, :20])
    c.sl[0], c.sl[1] = 1 << 20, -1
    out = kda.cache_evict(*c.args, 20, a, p, max_len=50)
    assert kda.last_device_error() == kda.KDA_ERR_INDEX and out.tolist() == [20, 0]


def test_evict_ignores_workspace_contents_and_stays_inside():
    for fill in (0, 255):
        c = Paged("bf16", [3000, 100], 2, 64, 16, seed=14)
        a, p = c.acc.clone(), c.pos.clone()
        size = kda.cache_evict_workspace_size(2, 2, 3000, 1000)
        ws = torch.full((size + 4096,), fill, dtype=torch.uint8, device=DEV)
        kda.cache_evict(*c.args, 1000, a, p, max_len=3000, workspace=ws[:size])
        assert (ws[size:] == fill).all()
        if fill == 0:
            first = (c.k.clone(), a, p)
    assert torch.equal(first[0].nan_to_num(), c.k.nan_to_num()) and torch.equal(first[1], a)
    assert torch.equal(first[2], p)


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_decode_loop_under_a_budget(io):
    """Serving as it runs: each step appends, attends with the gate and gathers weights; a cut to
    the budget follows every few steps. The cache, weights and positions are followed in fp64."""
    H, Hq, d, page, budget = 2, 8, 64, 16, 48
    c = Paged(io, [40, 47, 3, 0], H, d, page, room=30, seed=15)
    slots = c.max_pages * page
    c.acc = torch.zeros(4, H, slots, device=DEV)
    c.pos = torch.arange(slots, dtype=torch.int32, device=DEV).expand(4, H, -1).contiguous()
    K, V, A, P = f64(c.k), f64(c.v), f64(c.acc), f64(c.pos)
    lens, seen = list(c.lens), list(c.lens)
    table = c.table.numpy()
    for step in range(30):
        q, k, v, z = (c.rand(4, n, d) for n in (Hq, H, H, Hq))
        pos_dev = torch.tensor(seen, dtype=torch.int32, device=DEV)
        kda.cache_append(k.unsqueeze(1), v.unsqueeze(1), *c.args, positions=pos_dev, acc=c.acc,
                         pos=c.pos)
        ref.append(K, V, table, lens, f64(k), f64(v), [0, 1, 2, 3, 4], seen, A, P)
        c.sl += 1
        lens, seen = [x + 1 for x in lens], [x + 1 for x in seen]
        old = c.acc.clone()
        o = kda.paged_decode(q, *c.args, scale=0.2, z=z, acc=c.acc)
        c.lens = lens
        check_decode(c, q, o, 0.2, z, c.acc, old)
        A = f64(c.acc)                               # within its bound: the ranks go by it
        if step % 8 == 7:
            new = kda.cache_evict(*c.args, budget, c.acc, c.pos, n_first=2, n_recent=8,
                                  positions=torch.tensor(seen, dtype=torch.int32, device=DEV))
            lens = ref.evict(K, V, table, lens, budget, A, P, seen, 2, 8)
            c.sl = new
            assert new.tolist() == lens
        for n, m in enumerate(lens):
            p, r = ref.place(table, n, np.arange(m), page)
            assert np.array_equal(f64(c.k)[p, r], K[p, r]) and np.array_equal(f64(c.v)[p, r], V[p, r])
            assert np.array_equal(f64(c.pos)[n, :, :m], P[n, :, :m])
    assert kda.last_device_error() == kda.KDA_OK


def test_captured_step_follows_the_lengths():
    """One captured step (append, attend, evict), replayed while the lengths on the device grow."""
    H, Hq, d, page, budget = 2, 8, 128, 16, 30
    c = Paged("bf16", [10, 25], H, d, page, room=30, seed=16)
    slots = c.max_pages * page
    c.acc = torch.zeros(2, H, slots, device=DEV)
    c.pos = torch.zeros(2, H, slots, dtype=torch.int32, device=DEV)
    c.pos.copy_(torch.arange(slots, dtype=torch.int32, device=DEV))
    q, k, v = c.rand(2, Hq, d), c.rand(2, 1, H, d), c.rand(2, 1, H, d)
    o = torch.empty_like(q)
    seen = c.sl.clone()
    ws = torch.empty(max(kda.paged_decode_workspace_size(2, Hq, H, d, slots, True),
                         kda.cache_evict_workspace_size(2, H, slots, budget)),
                     dtype=torch.uint8, device=DEV)

    def step(c):
        kda.cache_append(k, v, *c.args, positions=seen, acc=c.acc, pos=c.pos)
        c.sl.add_(1)
        seen.add_(1)
        kda.paged_decode(q, *c.args, scale=0.1, acc=c.acc, o=o, workspace=ws)
        kda.cache_evict(*c.args, budget, c.acc, c.pos, positions=seen, n_recent=4, seqlens_out=c.sl,
                        workspace=ws)

    def twin():
        t = object.__new__(Paged)
        t.__dict__.update(c.__dict__)
        for name in ("k", "v", "sl", "acc", "pos"):
            setattr(t, name, getattr(c, name).clone())
        return t
    e = twin()                                     # the same steps without a graph
    seen0 = seen.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                  # a first call outside the capture, on a copy
        step(twin())
    torch.cuda.current_stream().wait_stream(side)
    seen.copy_(seen0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c)
    outs = []
    for i in range(12):
        q.copy_(c.rand(2, Hq, d)), k.copy_(c.rand(2, 1, H, d))
        seen_i = seen.clone()
        graph.replay()
        outs.append(o.clone())
        after = seen.clone()
        seen.copy_(seen_i)
        step(e)
        assert torch.equal(o, outs[-1]), i
        assert torch.equal(seen, after) and torch.equal(c.sl, e.sl)
    assert torch.equal(c.acc, e.acc) and torch.equal(c.pos, e.pos)
    assert torch.equal(c.k.nan_to_num(), e.k.nan_to_num())
    assert c.sl.tolist() == [22, 30]
    assert kda.last_device_error() == kda.KDA_OK


def test_c_entry_refuses_on_the_gpu_box_too():
    """A refused call launches nothing."""
    c = Paged("bf16", [20], 1, 64, 16)
    o = torch.full((1, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(kda.KdaError):
        kda.paged_decode(c.rand(1, 4, 64), *c.args, max_len=1000, o=o)
    with pytest.raises(kda.KdaError):
        kda.cache_evict(*c.args, 4, c.acc, c.pos, n_first=3, n_recent=2)
    assert (o == 5).all()


def test_c_entries_called_directly():
    """The C functions with single arguments do what the calls with packed ones do."""
    lib = kda.load_library()
    c = Paged("bf16", [70, 0, 33], 2, 64, 16, seed=3, room=4)
    q, z, new = c.rand(3, 4, 64), c.rand(3, 4, 64), c.rand(3, 2, 2, 64)
    k, v, acc, pos = (t.clone() for t in (c.k, c.v, c.acc, c.pos))
    ml = c.max_pages * c.page
    slots = c.slots
    p = [t.data_ptr() for t in (q, z, new, k, v, acc, pos, c.tab, c.sl)]
    stream = torch.cuda.current_stream().cuda_stream
    st = k.stride()[:3]
    pages = k.shape[0]
    sl2 = c.sl + 2
    o, out = torch.empty_like(q), torch.empty_like(c.sl)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    ml = min(ml, slots)
    cache = (p[3], p[4], *st, pages, 16, p[7], c.max_pages)
    assert lib.kda_cache_append(p[2], p[2], *cache, p[8], None, p[5], p[6], slots, None, None, 3, 2, 3,
                                2, 64, 1, stream) == kda.KDA_OK
    assert lib.kda_paged_decode(p[0], *cache, sl2.data_ptr(), p[1], 0.2, p[5], slots, o.data_ptr(), 3,
                                4, 2, 64, ml, 1, ws.data_ptr(), ws.numel(), stream) == kda.KDA_OK
    assert lib.kda_cache_evict(*cache, sl2.data_ptr(), None, 20, 2, 4, p[5], p[6], p[5], p[6], slots,
                               out.data_ptr(), 3, 2, 64, ml, 1, ws.data_ptr(), ws.numel(),
                               stream) == kda.KDA_OK
    kda.cache_append(new, new, *c.args, acc=c.acc, pos=c.pos)
    o2 = kda.paged_decode(q, c.k, c.v, c.tab, sl2, scale=0.2, z=z, acc=c.acc)
    out2 = kda.cache_evict(c.k, c.v, c.tab, sl2, 20, c.acc, c.pos, n_first=2, n_recent=4)
    assert kda.last_device_error() == kda.KDA_OK
    assert torch.equal(o, o2) and torch.equal(out, out2) and out.tolist() == [20, 2, 20]
    assert torch.equal(acc, c.acc) and torch.equal(pos, c.pos)
    assert torch.equal(k.nan_to_num(), c.k.nan_to_num()) and torch.equal(v.nan_to_num(), c.v.nan_to_num())
