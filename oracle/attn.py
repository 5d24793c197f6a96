"""Paged attention, plainly: the step maps, the cache write and attention row by row, in
float64 and Python integers.  Attention reads the visible keys alone."""
from __future__ import annotations

import numpy as np

TURN = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))


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


def tree_rows(ctx, new, tree_len, parents, window=0):
    """[(request, position, keys, their positions)] of every new token in a step with trees: the last tree_len[r] keys of
    request r are nodes, parents[r][i] the node that i follows or -1."""
    out = []
    for r, (c, m) in enumerate(zip(ctx, new)):
        n = int(tree_len[r])
        start = c + m - n
        path = []  # of every node: its ancestors, from the root, and itself
        for i in range(n):
            p = int(parents[r][i])
            path.append((path[p] if p >= 0 else []) + [i])
        for at in range(c, c + m):
            if at < start:
                keys = places = list(range(at + 1))
            else:
                keys = list(range(start)) + [start + i for i in path[at - start]]
                places = list(range(start + len(path[at - start])))
            pos = places[-1]
            seen = [(k, p) for k, p in zip(keys, places) if not window or pos - p < window]
            out.append((r, pos, np.array([k for k, _ in seen]), np.array([p for _, p in seen])))
    return out


def tree_attention(q, k_cache, v_cache, table, where, bt, scale, softcap=0.0, slopes=None, rows=None):
    """As `attention`, for the rows of `tree_rows`."""
    N, Hq, D = q.shape
    G = Hq // k_cache.shape[2]
    o, absum = np.zeros((N, Hq, D)), np.zeros((N, Hq, D))
    lse, xmax = np.full((N, Hq), -np.inf), np.zeros((N, Hq))
    for t, (r, pos, keys, places) in enumerate(where):
        blocks = np.asarray(table)[r if rows is None else rows[r], keys // bt]
        K, V = k_cache[blocks, keys % bt].astype(np.float64), v_cache[blocks, keys % bt].astype(np.float64)
        for h in range(Hq):
            x = scale * (K[:, h // G] @ q[t, h].astype(np.float64))
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if slopes is not None:
                x = x - float(slopes[h]) * (pos - places)
            m = x.max()
            e = np.exp(x - m)
            o[t, h] = e @ V[:, h // G] / e.sum()
            absum[t, h] = e @ np.abs(V[:, h // G]) / e.sum()
            lse[t, h] = m + np.log(e.sum())
            xmax[t, h] = np.abs(x).max()
    return o, lse, absum, xmax


def rotate(x, pos, inv_freq, axis=None, interleaved=False, scale=1.0, gain=None, eps=0.0):
    """Norms and rotation of heads x [N][H][D] at positions pos [axes][N]: (y, the sum of the magnitudes that make up each
    element of it)."""
    x = np.asarray(x, dtype=np.float64)
    if gain is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(gain, dtype=np.float64)
    n = len(inv_freq)
    y, mag = x.copy(), np.abs(x)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # (whole turns fall away before the product loses them)
        turns = np.asarray(pos)[0 if axis is None else axis[i]].astype(np.longdouble) * (np.longdouble(inv_freq[i]) / TURN)
        f = ((turns - np.floor(turns)) * TURN).astype(np.float64)[:, None]
        c, s = scale * np.cos(f), scale * np.sin(f)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        mag[..., a] = mag[..., b] = abs(scale) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, mag


def keep(cache, table, kv_len, tree_len, paths, bt, rows=None):
    """The cache [n_blocks][bt]... after the nodes paths[r] of each request's tree moved to the tree's start, and the
    lengths from there on."""
    out, ctx = cache.copy(), []
    for r, path in enumerate(paths):
        row, start = r if rows is None else rows[r], int(kv_len[r]) - int(tree_len[r])
        for i, node in enumerate(path):
            a, b = start + node, start + i
            out[table[row][b // bt], b % bt] = cache[table[row][a // bt], a % bt]
        ctx.append(start + len(path))
    return out, np.array(ctx)
