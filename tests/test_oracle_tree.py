"""Pins of the oracle's trees, rotations and kept paths."""
import math

import numpy as np

from oracle import attn as oa


def test_tree_rows_by_hand():
    # three cached tokens; of the tree 0 - 1, 0 - 2, 2 - 3 the first node is cached, too
    rows = oa.tree_rows([4], [3], [4], [[-1, 0, 0, 2]])
    assert [(p, k.tolist(), q.tolist()) for _, p, k, q in rows] == [
        (4, [0, 1, 2, 3, 4], [0, 1, 2, 3, 4]),
        (4, [0, 1, 2, 3, 5], [0, 1, 2, 3, 4]),
        (5, [0, 1, 2, 3, 5, 6], [0, 1, 2, 3, 4, 5])]
    rows = oa.tree_rows([4], [3], [4], [[-1, 0, 0, 2]], window=2)
    assert [k.tolist() for _, _, k, _ in rows] == [[3, 4], [3, 5], [5, 6]]


def test_a_chain_is_causal():
    rng = np.random.default_rng(0)
    K, V, q = rng.standard_normal((2, 16, 1, 8)), rng.standard_normal((2, 16, 1, 8)), rng.standard_normal((5, 2, 8))
    table = [[1, 0]]
    for window, slopes in ((0, None), (3, [0.5, 0.25])):
        a = oa.attention(q, K, V, table, oa.bounds([13], [5], window), 16, 0.3, 0.0, slopes)
        b = oa.tree_attention(q, K, V, table, oa.tree_rows([13], [5], [5], [[-1, 0, 1, 2, 3]], window), 16, 0.3, 0.0, slopes)
        for x, y in zip(a, b):
            assert np.allclose(x, y, rtol=1e-14, atol=1e-14)


def test_rotation_by_hand():
    x = np.array([[[3.0, 4.0, 1.0, 2.0, 7.0]]])
    quarter = [math.pi / 2, math.pi]
    y, mag = oa.rotate(x, [[1]], quarter)  # (3, 1) by a quarter, (4, 2) by a half
    assert np.allclose(y, [[[-1, -4, 3, -2, 7]]]) and np.allclose(mag, [[[4, 6, 4, 6, 7]]])
    y, _ = oa.rotate(x, [[0], [1]], quarter, axis=[1, 0], interleaved=True, scale=2.0)
    assert np.allclose(y, [[[-8, 6, 2, 4, 7]]])
    y, _ = oa.rotate(x, [[1 << 30]], [2 * math.pi / 4] * 2)  # a whole number of turns
    assert np.allclose(y, x, atol=1e-6)
    y, _ = oa.rotate(x, [[0]], [], gain=[1, 1, 1, 1, 2], eps=1.0)
    assert np.allclose(y, x / math.sqrt(79 / 5 + 1) * [1, 1, 1, 1, 2])


def test_keep_by_hand():
    cache = np.arange(32).reshape(2, 16)
    out, ctx = oa.keep(cache, [[1, 0]], [20], [6], [[0, 2, 5]], 16)
    # keys 14 .. 19; 16 -> 15, 19 -> 16
    want = cache.copy()
    want[1, 15], want[0, 0] = cache[0, 0], cache[0, 3]
    assert np.array_equal(out, want) and ctx.tolist() == [17]
