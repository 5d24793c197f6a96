"""The paged-attention oracle on hand-worked cases and against a per-element restatement."""
import math

import numpy as np
import pytest

from oracle import attn as oa


def test_step_maps_by_hand():
    # blocks of 4: request 0 holds 5 tokens in blocks 7, 2 and adds 4 (opens one), request 1 is new with 1
    table = -np.ones((3, 3), dtype=int)
    table[0, :2] = [7, 2]
    got = oa.step_maps([5, 0], [4, 1], 4, [9, 3], table, rows=[0, 2], n_tokens=7)
    assert got[0].tolist() == [[7, 2, 9], [-1, -1, -1], [3, -1, -1]]
    assert got[1].tolist() == [0, 4, 5] and got[2].tolist() == [9, 1]
    assert got[3].tolist() == [9, 10, 11, 36, 12, -1, -1]
    assert got[4].tolist() == [5, 6, 7, 8, 0, -1, -1]


def test_bounds_by_hand():
    assert oa.bounds([3], [2]) == [(0, 3, 0, 4), (0, 4, 0, 5)]
    assert oa.bounds([3], [2], window=2) == [(0, 3, 2, 4), (0, 4, 3, 5)]
    assert oa.bounds([0], [3], doc_start=[0, 1, 1], bidir_len=[2]) == [(0, 0, 0, 2), (0, 1, 1, 2), (0, 2, 1, 3)]
    assert oa.bounds([1, 0], [0, 1]) == [(1, 0, 0, 1)]


@pytest.mark.parametrize("softcap,alibi", [(0.0, False), (2.0, False), (0.0, True), (2.0, True)])
def test_attention_against_elements(softcap, alibi):
    rng = np.random.default_rng(3)
    bt, D, Hq, Hkv = 4, 8, 4, 2
    k, v = rng.normal(size=(2, 5, bt, Hkv, D))
    q = rng.normal(size=(3, Hq, D))
    table = np.array([[4, 1, 0]])
    where = oa.bounds([6], [3], window=5)
    slopes = np.array([0.5, 0.25, 0.125, 1.0]) if alibi else None
    o, lse, _, _ = oa.attention(q, k, v, table, where, bt, 0.3, softcap, slopes)
    for t, (_, p, lo, hi) in enumerate(where):
        for h in range(Hq):
            num, den = [0.0] * D, 0.0
            for j in range(lo, hi):
                b, i = int(table[0, j // bt]), j % bt
                x = 0.3 * math.fsum(q[t, h, d] * k[b, i, h // 2, d] for d in range(D))
                if softcap:
                    x = softcap * math.tanh(x / softcap)
                if alibi:
                    x -= slopes[h] * abs(p - j)
                den += math.exp(x)
                num = [n + math.exp(x) * v[b, i, h // 2, d] for d, n in enumerate(num)]
            assert np.allclose(o[t, h], np.array(num) / den, rtol=1e-12, atol=1e-14)
            assert abs(lse[t, h] - math.log(den)) < 1e-12


def test_a_row_without_keys_is_zero():
    z = np.zeros((1, 4, 1, 8))
    o, lse, _, _ = oa.attention(np.ones((1, 1, 8)), z, z, [[0]], [(0, 0, 0, 0)], 4, 1.0)
    assert not o.any() and np.isneginf(lse).all()


def test_append_by_hand():
    cache = np.zeros((2, 4, 1, 2))
    oa.append(cache, np.arange(6).reshape(3, 1, 2), [5, -1, 2])
    assert cache[1, 1, 0].tolist() == [0, 1] and cache[0, 2, 0].tolist() == [4, 5] and cache.sum() == 10
