"""The library keeps nothing of a CUDA context: its calls work in the next one too."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import ctypes
import numpy as np
from kimi_delta_attention_32_b200 import kda

lib = kda.load_library()          # its runtime's functions are reached through it too
N, H, d, page, length = 3, 2, 128, 16, 40


def up(x):
    p = ctypes.c_void_p()
    assert lib.cudaMalloc(ctypes.byref(p), ctypes.c_size_t(x.nbytes)) == 0
    assert lib.cudaMemcpy(p, ctypes.c_void_p(x.ctypes.data), ctypes.c_size_t(x.nbytes), 1) == 0
    return p


def down(p, like):
    x = np.empty_like(like)
    assert lib.cudaMemcpy(ctypes.c_void_p(x.ctypes.data), p, ctypes.c_size_t(x.nbytes), 2) == 0
    return x


def steps():
    g = np.random.default_rng(1)
    k, v = (g.standard_normal((9, page, H, d), dtype=np.float32) for _ in range(2))
    q, new = g.standard_normal((N, H, d), dtype=np.float32), np.ones((N, H, d), np.float32)
    table = np.arange(9, dtype=np.int32).reshape(N, 3)
    lens, acc = np.full(N, length, np.int32), np.zeros((N, H, 48), np.float32)
    kd, vd, qd, nd, td, ld, ad, od = map(up, (k, v, q, new, table, lens, acc, q))
    pd, wd = up(acc.view(np.int32)), up(np.zeros(1 << 25, np.uint8))
    cache = (kd, vd, page * H * d, H * d, d, 9, page, td, 3)
    assert lib.kda_cache_append(nd, nd, *cache, ld, None, ad, pd, 48, None, None, N, 1, N, H, d, 0,
                                None) == 0
    assert lib.kda_paged_decode(qd, *cache, ld, None, 0.1, ad, 48, od, N, H, H, d, 48, 0, wd, 1 << 25,
                                None) == 0
    assert lib.kda_cache_evict(*cache, ld, None, 20, 0, 0, ad, pd, ad, pd, 48, ld, N, H, d, 48, 0, wd,
                               1 << 25, None) == 0
    assert lib.kda_last_device_error(None) == kda.KDA_OK
    o = down(od, q)
    assert (down(ld, lens) == 20).all()
    K, V = (x.reshape(N, 48, H, d)[:, :length].astype(np.float64) for x in (k, v))
    s = np.einsum("nhd,nshd->nhs", q, K) * 0.1
    w = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("nhs,nshd->nhd", w / w.sum(-1, keepdims=True), V)
    # 256 fp32 operations a sum at most, of weights that add up to 1 and values below 6
    assert np.abs(o - want).max() < 256 * 6 * 2.0 ** -23
    # a length beyond the table is reported
    assert lib.cudaMemcpy(ld, ctypes.c_void_p(np.full(N, 49, np.int32).ctypes.data),
                          ctypes.c_size_t(4 * N), 1) == 0
    assert lib.kda_paged_decode(qd, *cache, ld, None, 0.1, None, 0, od, N, H, H, d, 48, 0, wd, 1 << 25,
                                None) == 0
    assert lib.kda_last_device_error(None) == kda.KDA_ERR_INDEX


for _ in range(3):
    steps()
    assert lib.cudaDeviceReset() == 0
print("done")
"""


def test_calls_work_after_the_context_is_replaced():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, timeout=300, capture_output=True,
                       text=True)
    assert r.returncode == 0 and r.stdout == "done\n", r.stdout + r.stderr
