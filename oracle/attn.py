"""Paged attention, plainly: the step maps, the cache write and attention row by row, in
float64 and Python integers.  Attention reads the visible keys alone."""
from __future__ import annotations

import numpy as np


def step_maps(ctx, new, bt, new_ids, table, rows=None, n_tokens=None):
    """(table, q_start, kv_len, slot, pos) of a step; ``table`` is copied, slots and positions of
    rows past the last new token are -1."""
    table = np.array(table, dtype=np.int64)
    n = int(sum(new)) if n_tokens is None else n_tokens
    slot, pos = [-1] * n, [-1] * n
    q_start, kv_len, t, used = [0], [], 0, 0
    for r, (c, m) in enumerate(zip(ctx, new)):
        row = r if rows is None else rows[r]
        for page in range(-(-c // bt), -(-(c + m) // bt)):
            table[row, page] = new_ids[used]
            used += 1
        for p in range(c, c + m):
            slot[t], pos[t] = int(table[row, p // bt]) * bt + p % bt, p
            t += 1
        q_start.append(t)
        kv_len.append(c + m)
    return table, np.array(q_start), np.array(kv_len), np.array(slot), np.array(pos)


def append(cache, rows, slot):
    """cache [n_blocks][bt][H][D] (changed in place) with rows [N][H][D] at their slots."""
    bt = cache.shape[1]
    for t, s in enumerate(slot):
        if s >= 0:
            cache[s // bt, s % bt] = rows[t]


def bounds(ctx, new, window=0, doc_start=None, bidir_len=None):
    """[(request, position, lo, hi)] of every new token."""
    out, t = [], 0
    for r, (c, m) in enumerate(zip(ctx, new)):
        for p in range(c, c + m):
            lo = max(0, p - window + 1) if window else 0
            if doc_start is not None:
                lo = max(lo, int(doc_start[t]))
            hi = p + 1 if bidir_len is None else max(p + 1, int(bidir_len[r]))
            out.append((r, p, lo, min(c + m, hi)))
            t += 1
    return out


def attention(q, k_cache, v_cache, table, where, bt, scale, softcap=0.0, slopes=None, rows=None):
    """o [N][Hq][D], lse [N][Hq] and absum [N][Hq][D] = sum_j p_j |v_j| (what rounding errors of the
    probabilities scale with), xmax [N][Hq] the largest |score|."""
    N, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    G = Hq // Hkv
    o, absum = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse, xmax = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    for t, (r, p, lo, hi) in enumerate(where):
        if lo >= hi:
            continue
        j = np.arange(lo, hi)
        blocks = np.asarray(table)[r if rows is None else rows[r], j // bt]
        K, V = k_cache[blocks, j % bt].astype(np.float64), v_cache[blocks, j % bt].astype(np.float64)
        for h in range(Hq):
            x = scale * (K[:, h // G] @ q[t, h].astype(np.float64))
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                x = x - float(slopes[h]) * np.abs(p - j)
            m = x.max()
            e = np.exp(x - m)
            o[t, h] = e @ V[:, h // G] / e.sum()
            absum[t, h] = e @ np.abs(V[:, h // G]) / e.sum()
            lse[t, h] = m + np.log(e.sum())
            xmax[t, h] = np.abs(x).max()
    return o, lse, absum, xmax
