"""CPU tests of the paged cache's entry points: the C ABI's and the binding's refusals, and the
workspace queries."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from kimi_delta_attention_32_b200 import build as kbuild
from kimi_delta_attention_32_b200 import kda
from test_abi import FAKE, MIS, ROOT, _cu_host

INV, UNS, WS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
ODD = ctypes.c_void_p(0x10002)           # not even 4-byte aligned


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


CACHE = dict(kc=FAKE, vc=FAKE, ps=16 * 2 * 128, ss=2 * 128, hs=128, np=8, page=16, bt=FAKE, mp=4)


def _append(lib, **kw):
    a = dict(CACHE, k=FAKE, v=FAKE, sl=FAKE, po=None, acc=None, pos=None, slots=0, cu=None, cuh=None,
             B=2, T=1, N=0, H=2, d=128, io=1)
    a.update(kw)
    return lib.kda_cache_append(a["k"], a["v"], a["kc"], a["vc"], a["ps"], a["ss"], a["hs"], a["np"],
                                a["page"], a["bt"], a["mp"], a["sl"], a["po"], a["acc"], a["pos"],
                                a["slots"], a["cu"], a["cuh"], a["B"], a["T"], a["N"], a["H"],
                                a["d"], a["io"], None)


def _decode(lib, **kw):
    a = dict(CACHE, q=FAKE, sl=FAKE, z=None, scale=1.0, acc=None, slots=0, o=FAKE, N=2, Hq=8, H=2,
             d=128, ml=64, io=1, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.kda_paged_decode(a["q"], a["kc"], a["vc"], a["ps"], a["ss"], a["hs"], a["np"],
                                a["page"], a["bt"], a["mp"], a["sl"], a["z"], a["scale"], a["acc"],
                                a["slots"], a["o"], a["N"], a["Hq"], a["H"], a["d"], a["ml"],
                                a["io"], a["ws"], a["wsb"], None)


def _evict(lib, **kw):
    a = dict(CACHE, sl=FAKE, po=None, keep=32, nf=4, nr=8, acc=FAKE, pos=FAKE, ao=FAKE, qo=FAKE,
             slots=64, so=FAKE, N=2, H=2, d=128, ml=64, io=1, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    return lib.kda_cache_evict(a["kc"], a["vc"], a["ps"], a["ss"], a["hs"], a["np"], a["page"],
                               a["bt"], a["mp"], a["sl"], a["po"], a["keep"], a["nf"], a["nr"],
                               a["acc"], a["pos"], a["ao"], a["qo"], a["slots"], a["so"], a["N"],
                               a["H"], a["d"], a["ml"], a["io"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fn", [_append, _decode, _evict])
@pytest.mark.parametrize("kw,status", [
    (dict(kc=None), INV), (dict(vc=MIS), INV), (dict(bt=None), INV), (dict(bt=ODD), INV),
    (dict(sl=None), INV), (dict(sl=ODD), INV), (dict(page=0), INV), (dict(np=-1), INV),
    (dict(mp=-1), INV), (dict(H=0), INV), (dict(d=0), INV), (dict(io=7), INV),
    (dict(ps=0), INV), (dict(ss=-256), INV), (dict(hs=64), INV),       # strides below d
    (dict(hs=129), INV),                                               # not 16 bytes
    (dict(io=0, ss=258), INV),
    (dict(d=96, hs=96), UNS), (dict(d=32), UNS), (dict(mp=1 << 30), UNS),
])
def test_cache_arguments_are_checked(lib, fn, kw, status):
    assert fn(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INV), (dict(v=MIS), INV), (dict(po=ODD), INV), (dict(acc=FAKE), INV),
    (dict(pos=FAKE, slots=0), INV), (dict(slots=-1), INV), (dict(acc=ODD, slots=8), INV),
    (dict(B=-1), INV), (dict(B=1 << 16, T=1 << 16), UNS), (dict(cu=FAKE), INV),
])
def test_append_refuses(lib, kw, status):
    assert _append(lib, **kw) == status


def test_append_refuses_bad_cu_seqlens(lib):
    keep, cuh = _cu_host([0, 3, 2])
    assert _append(lib, cu=FAKE, cuh=cuh, N=2) == INV
    keep2, cuh = _cu_host([1, 2, 3])
    assert _append(lib, cu=FAKE, cuh=cuh, N=2) == INV
    del keep, keep2


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INV), (dict(o=MIS), INV), (dict(z=MIS), INV), (dict(Hq=7), INV), (dict(Hq=0), INV),
    (dict(N=-1), INV), (dict(ml=-1), INV), (dict(ml=65), INV),         # beyond the block table
    (dict(acc=FAKE), INV), (dict(acc=FAKE, slots=63), INV), (dict(acc=ODD, slots=64), INV),
    (dict(ws=None), WS), (dict(ws=MIS), WS),
    (dict(N=1 << 15, H=1, Hq=1 << 17), UNS),                           # N * Hq counts blocks
])
def test_decode_refuses(lib, kw, status):
    assert _decode(lib, **kw) == status


def test_decode_refuses_a_short_workspace(lib):
    out = ctypes.c_size_t(0)
    for with_acc in (0, 1):
        assert lib.kda_paged_decode_workspace_size(2, 8, 2, 128, 64, with_acc, ctypes.byref(out)) == 0
        kw = dict(acc=FAKE, slots=64) if with_acc else {}
        assert _decode(lib, wsb=out.value - 1, **kw) == WS


@pytest.mark.parametrize("kw,status", [
    (dict(acc=None), INV), (dict(pos=None), INV), (dict(ao=None), INV), (dict(qo=None), INV),
    (dict(so=None), INV), (dict(so=ODD), INV), (dict(po=ODD), INV),
    (dict(keep=-1), INV), (dict(nf=-1), INV), (dict(nr=-1), INV), (dict(nf=25, nr=8), INV),
    (dict(nf=2 ** 31 - 1, nr=2 ** 31 - 1), INV),
    (dict(ml=65, slots=100), INV), (dict(ml=64, slots=63), INV), (dict(ml=-1), INV),
    (dict(ao=ctypes.c_void_p(0x10000 + 64)), INV),                     # overlaps acc in part
    (dict(qo=ctypes.c_void_p(0x10000 - 64)), INV),
    (dict(ws=MIS), WS), (dict(wsb=3), WS),
])
def test_evict_refuses(lib, kw, status):
    assert _evict(lib, **kw) == status


def test_workspace_queries(lib):
    out = ctypes.c_size_t(0)
    size = lib.kda_paged_decode_workspace_size
    assert size(4, 32, 8, 128, 1000, 0, None) == INV
    assert size(4, 32, 7, 128, 1000, 0, ctypes.byref(out)) == INV
    assert size(-1, 32, 8, 128, 1000, 0, ctypes.byref(out)) == INV
    assert size(4, 32, 8, 128, -1, 0, ctypes.byref(out)) == INV
    assert size(2 ** 30, 2 ** 30, 1, 128, 2 ** 30, 1, ctypes.byref(out)) == UNS    # over 2^63 bytes
    assert size(4, 32, 8, 128, 1000, 0, ctypes.byref(out)) == 0
    plain = out.value
    assert size(4, 32, 8, 128, 1000, 1, ctypes.byref(out)) == 0
    assert out.value >= plain
    size = lib.kda_cache_evict_workspace_size
    assert size(4, 8, 1000, -1, ctypes.byref(out)) == INV
    assert size(4, 0, 1000, 10, ctypes.byref(out)) == INV
    assert size(4, 8, 1000, 400, None) == INV
    assert size(4, 8, 1000, 400, ctypes.byref(out)) == 0


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_split_covers_every_tile_once(tmp_path):
    """The division of tiles over blocks: contiguous, complete, none empty, sizes one apart at
    most, and split_block_of is its inverse."""
    src = tmp_path / "split.cpp"
    src.write_text(r"""
#include "decode_split.h"
using namespace kda;
int main() {
    const int64_t works[] = {1, 2, 3, 7, 147, 148, 149, 295, 296, 297, 320, 1000, 12345, 65536,
                             131072, 1 << 20, (1ll << 40) + 12345};
    const int mosts[] = {1, 2, 37, 148, 160, 296, 320};
    for (int64_t W : works)
        for (int most : mosts) {
            const int C = split_blocks(W, most);
            if (C < 1 || C > most || C > W) return 1;
            if (split_begin(W, C, 0) != 0 || split_begin(W, C, C) != W) return 2;
            for (int c = 0; c < C; ++c) {
                const int64_t a = split_begin(W, C, c), b = split_begin(W, C, c + 1);
                if (b - a < W / C || b - a > W / C + 1 || b <= a) return 3;
                if (split_block_of(W, C, a) != c || split_block_of(W, C, b - 1) != c ||
                    split_block_of(W, C, a + (b - a) / 2) != c) return 4;
            }
        }
    return 0;
}
""")
    exe = tmp_path / "split"
    inc = os.path.join(ROOT, "kimi_delta_attention_32_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", inc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0


def test_index_status_has_a_text(lib):
    assert kda.KDA_ERR_INDEX == 6 and b"out of range" in lib.kda_status_string(6)


def _tensors(io=torch.bfloat16, N=2, H=2, d=128, page=16, pages=8):
    c = torch.zeros(pages, page, H, d, dtype=io)
    i32 = dict(dtype=torch.int32)
    return dict(k_cache=c, v_cache=c.clone(), block_table=torch.zeros(N, 4, **i32),
                seqlens=torch.zeros(N, **i32))


def test_binding_refuses():
    """The binding's checks come before any call; tensors on the host are refused last."""
    t = _tensors()
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    ws = torch.zeros(16, dtype=torch.uint8)

    def dec(q=q, **kw):
        a = dict(t, workspace=ws)
        a.update(kw)
        return kda.paged_decode(q, **a)
    with pytest.raises(ValueError, match="CUDA tensor"):
        dec()
    with pytest.raises(TypeError):
        dec(q=q.float())
    with pytest.raises(ValueError, match="contiguous"):
        dec(q=torch.zeros(8, 2, 128, dtype=torch.bfloat16).transpose(0, 1))
    with pytest.raises(ValueError, match="shape"):
        dec(q=q[:1])
    with pytest.raises(ValueError, match="shape"):
        dec(seqlens=t["seqlens"][:1])
    with pytest.raises(TypeError):
        dec(block_table=t["block_table"].long())
    with pytest.raises(ValueError, match="stride"):
        dec(v_cache=t["v_cache"].transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="stride"):
        dec(k_cache=torch.zeros(8, 16, 2, 256, dtype=torch.bfloat16)[..., ::2],
            v_cache=torch.zeros(8, 16, 2, 256, dtype=torch.bfloat16)[..., ::2])
    with pytest.raises(ValueError):
        dec(v_cache=t["v_cache"][:4])
    with pytest.raises(TypeError):
        dec(k_cache=t["k_cache"].half(), v_cache=t["v_cache"].half())
    with pytest.raises(ValueError, match="workspace"):
        dec(workspace=torch.zeros(16))
    with pytest.raises(TypeError):
        dec(acc=torch.zeros(2, 2, 64, dtype=torch.float64))
    k = torch.zeros(2, 1, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.cache_append(k, k, **t)
    with pytest.raises(ValueError, match="sequences"):
        kda.cache_append(k[:1], k[:1], **t)
    with pytest.raises(ValueError):
        kda.cache_append(k[:, 0], k[:, 0], **t)          # packed without cu_seqlens
    with pytest.raises(ValueError, match="cu_host"):
        kda.cache_append(k[:, 0], k[:, 0], cu_seqlens=torch.zeros(3, dtype=torch.int32), **t)
    acc, pos = torch.zeros(2, 2, 64), torch.zeros(2, 2, 64, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        kda.cache_evict(keep=8, acc=acc, pos=pos, workspace=ws, **t)
    with pytest.raises(ValueError, match="shape"):
        kda.cache_evict(keep=8, acc=acc, pos=pos[:, :, :32], workspace=ws, **t)
    with pytest.raises(ValueError, match="int32"):
        kda.cache_evict(keep=(1 << 32) + 8, acc=acc, pos=pos, workspace=ws, **t)
    with pytest.raises(ValueError, match="int32"):
        dec(max_len=1 << 32)
    with pytest.raises(TypeError, match="required"):
        kda.cache_evict(keep=8, acc=acc, pos=None, workspace=ws, **t)


class _Words:
    """The library with each call's arguments passed as words."""

    def __init__(self, lib):
        self.lib = lib

    def _call(self, function, args):
        which, pack = function
        args = [a if a is None or isinstance(a, (int, float)) else
                ctypes.cast(a, ctypes.c_void_p).value for a in args]
        return self.lib.kda_paged_call(which, pack(*(a or 0 for a in args)), len(args))

    def kda_cache_append(self, *a):
        return self._call(kda._APPEND, a)

    def kda_paged_decode(self, *a):
        return self._call(kda._DECODE, a)

    def kda_cache_evict(self, *a):
        return self._call(kda._EVICT, a)


@pytest.mark.parametrize("fn", [_append, _decode, _evict])
def test_words_reach_the_same_checks(lib, fn):
    """One argument wrong at a time, the direct call and the one with words refuse it alike."""
    by_word = _Words(lib)
    for kw in (dict(kc=None), dict(vc=MIS), dict(ps=-8), dict(ss=4), dict(hs=12), dict(np=-1),
               dict(page=0), dict(bt=ODD), dict(mp=-1), dict(sl=None), dict(H=0),
               dict(d=96), dict(io=7), dict(mp=1 << 28, page=64)):
        want = fn(lib, **kw)
        assert want in (INV, UNS), kw
        assert fn(by_word, **kw) == want, kw
    assert _decode(by_word, wsb=0) == _evict(by_word, ws=None) == WS
    assert _decode(by_word, Hq=7) == _evict(by_word, nf=30, nr=8) == INV
    assert _append(by_word, k=None) == _append(by_word, po=ODD) == INV


@pytest.mark.parametrize("fn,ints", [
    (_append, ("np", "page", "mp", "slots", "B", "T", "N", "H", "d", "io")),
    (_decode, ("np", "page", "mp", "slots", "N", "Hq", "H", "d", "ml", "io")),
    (_evict, ("np", "page", "mp", "keep", "nf", "nr", "slots", "N", "H", "d", "ml", "io"))])
def test_words_wider_than_an_int_are_refused(lib, fn, ints):
    """2^32 more than a size that would be taken is not cut to it. (d = 96 ends the good call.)"""
    by_word = _Words(lib)
    good = dict(np=8, page=16, mp=4, slots=64, B=2, T=1, N=2, H=2, d=96, io=1, Hq=8, ml=64, keep=32,
                nf=4, nr=8)
    assert fn(by_word, d=96) == UNS
    for x in ints:
        for far in (1 << 32, -(1 << 32)):
            assert fn(by_word, **{"d": 96, x: good[x] + far}) == INV, x


def test_words_refusals(lib):
    for (which, pack), n in ((kda._APPEND, 25), (kda._DECODE, 25), (kda._EVICT, 28)):
        words = pack(*[0] * n)
        assert lib.kda_paged_call(which, words, n) == INV        # no cache
        assert lib.kda_paged_call(which, words, n - 1) == INV
        assert lib.kda_paged_call(which, words + words, n + 1) == INV
        assert lib.kda_paged_call(which, None, n) == INV
    assert lib.kda_paged_call(3, bytes(8 * 28), 28) == INV
    assert lib.kda_paged_call(-1, bytes(8 * 28), 28) == INV
