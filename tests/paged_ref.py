"""The paged cache's operators in fp64 on the host (numpy), sequence by sequence, and the error
bounds of the device's arithmetic.

    append: token i of sequence n -> slot len_n + i, acc 0, pos seen_n + i
    decode: s_j = scale q . K_j, w = softmax(s), o = (sum_j w_j V_j) sigmoid(z), acc_j += sum w_j
    evict:  the keep best of (guarded, acc, -slot) stay; those behind slot keep fill the free
            slots before it, both in slot order
"""
from __future__ import annotations

import numpy as np

U24, HALF = 2.0 ** -24, {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # fp32's and each type's half step


def place(table, n, slots, page):
    """(page, row) of slots of sequence n."""
    slots = np.asarray(slots, dtype=np.int64)
    return table[n, slots // page], slots % page


def append(k_cache, v_cache, table, lens, k, v, cu, seen=None, acc=None, pos=None):
    """In place on numpy arrays [pages, page, H, d]; k, v packed [T, H, d]."""
    page = k_cache.shape[1]
    seen = lens if seen is None else seen
    for n in range(len(lens)):
        m = cu[n + 1] - cu[n]
        p, r = place(table, n, lens[n] + np.arange(m), page)
        k_cache[p, r], v_cache[p, r] = k[cu[n]:cu[n + 1]], v[cu[n]:cu[n + 1]]
        if acc is not None:
            acc[n, :, lens[n]:lens[n] + m] = 0
        if pos is not None:
            pos[n, :, lens[n]:lens[n] + m] = seen[n] + np.arange(m)


def decode(q, k_cache, v_cache, table, lens, scale, z=None, skip=None):
    """(o, weights per sequence [Hkv, len], sum_j w_j |V_j|, relative error of the weights and
    sums in the device's fp32). skip(page numbers) -> True for slots to leave out. fp64 numpy in and
    out."""
    N, Hq, d = q.shape
    H = k_cache.shape[2]
    G, page = Hq // H, k_cache.shape[1]
    o = np.zeros((N, Hq, d))
    mag = np.zeros((N, Hq, d))
    rel = np.zeros((N, Hq, 1))
    weights = []
    for n in range(N):
        j = np.arange(lens[n])
        if skip is not None and lens[n]:
            j = j[~skip(table[n, j // page])]
        w_n = np.zeros((H, lens[n]))
        for h in range(H if len(j) else 0):
            p, r = place(table, n, j, page)
            K, V = k_cache[p, r, h], v_cache[p, r, h]
            for g in range(G):
                x = q[n, h * G + g]
                s = K @ x * scale
                w = np.exp(s - s.max())
                w /= w.sum()
                w_n[h, j] += w
                o[n, h * G + g] = w @ V
                mag[n, h * G + g] = w @ np.abs(V)
                # score error: d products and sums in fp32 (operands at most 3 x 2^-22 off), the
                # scale, and the exponential's argument and result (2^-21)
                ds = (d + 24) * U24 * 2 * np.abs(scale) * (np.abs(K) @ np.abs(x)).max() + \
                    np.abs(s).max() * 4 * U24 + 2.0 ** -21
                # weights move by at most exp(2 ds) - 1; the sums over len add len 2^-24 each
                rel[n, h * G + g] = np.expm1(2 * ds) + 2 * (len(j) + 16) * U24
        weights.append(w_n)
    if z is not None:
        gate = 1 / (1 + np.exp(-z))
        o, mag = o * gate, mag * gate
        rel = rel + 2.0 ** -21
    return o, weights, mag, rel


def decode_bound(io, o, mag, rel):
    """Elementwise bound: the weights as the sum of two bf16 (2^-16; fp32 splits lie below that),
    the output rounded to the io type (half a step), beside the fp32 part."""
    return (2.0 ** -16 + rel) * mag + HALF[io] * (np.abs(o) + (2.0 ** -16 + rel) * mag) + 1e-30


def evict(k_cache, v_cache, table, lens, keep, acc, pos, seen, n_first, n_recent):
    """In place on all arrays; returns the new lengths."""
    page = k_cache.shape[1]
    out = []
    for n in range(len(lens)):
        length = int(lens[n])
        out.append(min(length, keep))
        if length <= keep:
            continue
        for h in range(acc.shape[1]):
            a, p = acc[n, h, :length].astype(np.float64), pos[n, h, :length]
            rank = []
            for s in range(length):
                guarded = p[s] < n_first or p[s] >= seen[n] - n_recent
                nan = np.isnan(a[s])
                rank.append((0 if guarded else 2 if nan else 1,
                             0.0 if guarded or nan else -a[s], s))
            kept = {x[2] for x in sorted(rank)[:keep]}
            holes = [s for s in range(keep) if s not in kept]
            tails = [s for s in range(keep, length) if s in kept]
            assert len(holes) == len(tails)
            for to, frm in zip(holes, tails):
                (p1, r1), (p2, r2) = place(table, n, to, page), place(table, n, frm, page)
                k_cache[p1, r1, h], v_cache[p1, r1, h] = k_cache[p2, r2, h], v_cache[p2, r2, h]
                acc[n, h, to], pos[n, h, to] = acc[n, h, frm], pos[n, h, frm]
    return out
