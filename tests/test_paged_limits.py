"""The size limits that the header states for the paged cache's calls, and the division of tiles at
every block count that a GPU can have."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import pytest

from kimi_delta_attention_32_b200 import kda
from test_abi import ROOT
from test_paged_abi import UNS, lib      # noqa: F401

OK = kda.KDA_OK


@pytest.mark.parametrize("N,ml,status", [
    (64, 1 << 30, OK), (1 << 20, 1 << 16, OK), ((1 << 30) - 1, 64, OK), (1 << 30, 64, UNS),
    ((1 << 31) - 1, 63, OK), (128, (1 << 30) - 128, OK), (128, 1 << 30, UNS)])
def test_decode_counts_tiles_in_31_bits(lib, N, ml, status):       # noqa: F811
    """N (max_len / 64 + 1) < 2^31."""
    assert (N * (ml // 64 + 1) < 1 << 31) == (status == OK)
    out = ctypes.c_size_t(0)
    assert lib.kda_paged_decode_workspace_size(N, 1, 1, 128, ml, 0, ctypes.byref(out)) == status


def test_decode_workspace_with_weights(lib):       # noqa: F811
    """A score of 4 bytes a query head and slot of the bound, beside some megabytes."""
    out = ctypes.c_size_t(0)
    for N, Hq, H, ml in ((1, 32, 8, 200), (256, 32, 8, 131072), (4, 12, 1, 5000)):
        assert lib.kda_paged_decode_workspace_size(N, Hq, H, 128, ml, 0, ctypes.byref(out)) == OK
        plain = out.value
        assert plain < 20 << 20
        assert lib.kda_paged_decode_workspace_size(N, Hq, H, 128, ml, 1, ctypes.byref(out)) == OK
        scores = 4 * N * Hq * (-(-ml // 128) * 128)
        assert scores <= out.value - plain <= 4 * scores + 64 * (N * Hq + 64)


@pytest.mark.parametrize("N,H,ml,keep,status", [
    (64, 8, 1 << 30, 1 << 29, UNS), (64, 8, 1 << 28, 1 << 27, OK), (64, 8, 1 << 30, 1 << 22, OK),
    (64, 8, 1 << 30, (1 << 30) - (1 << 22), OK), (1 << 28, 1, 64, 32, UNS), ((1 << 28) - 1, 1, 64, 32, OK)])
def test_evict_counts_blocks_in_31_bits(lib, N, H, ml, keep, status):       # noqa: F811
    """8 N Hkv < 2^31 and N Hkv ceil(min(keep, max_len - keep) / 64) < 2^31."""
    most = min(keep, ml - keep)
    assert (8 * N * H < 1 << 31 and N * H * -(-most // 64) < 1 << 31) == (status == OK)
    out = ctypes.c_size_t(0)
    assert lib.kda_cache_evict_workspace_size(N, H, ml, keep, ctypes.byref(out)) == status
    if status == OK:
        assert out.value == 4 * N * H * (2 * most + 1)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_split_at_every_block_count(tmp_path):
    """Contiguous, complete, none empty, sizes one apart at most, and split_block_of the inverse, for 1
    to 480 blocks (three an SM of 160)."""
    src = tmp_path / "split.cpp"
    src.write_text(r"""
#include "decode_split.h"
using namespace kda;
int main() {
    const int64_t works[] = {1, 2, 5, 147, 295, 296, 297, 443, 444, 445, 479, 480, 481, 1000, 65536,
                             (1ll << 31) - 1, (1ll << 31), (1ll << 40) + 12345};
    for (int64_t W : works)
        for (int most = 1; most <= 480; ++most) {
            const int C = split_blocks(W, most);
            if (C < 1 || C > most || C > W) return 1;
            if (split_begin(W, C, 0) != 0 || split_begin(W, C, C) != W) return 2;
            for (int c = 0; c < C; ++c) {
                const int64_t a = split_begin(W, C, c), b = split_begin(W, C, c + 1);
                if (b - a < W / C || b - a > W / C + 1 || b <= a) return 3;
                if (split_block_of(W, C, a) != c || split_block_of(W, C, b - 1) != c) return 4;
            }
        }
    return 0;
}
""")
    exe = tmp_path / "split"
    inc = os.path.join(ROOT, "kimi_delta_attention_32_b200", "csrc")
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", inc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
