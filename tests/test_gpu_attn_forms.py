"""Paged attention in the shapes between the forms' limits: head groups of every size, shared prefixes in all
forms and types, caches whose rows L2 fetches in small parts, and numbers near the ends of their range."""
import numpy as np
import pytest

from attn_helpers import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


@pytest.mark.parametrize("Hq,Hkv", [(128, 1), (96, 2), (40, 2), (17, 1), (16, 1), (15, 3), (10, 2), (64, 64)])
@pytest.mark.parametrize("ctx,new", [([0, 15, 130, 700], [1, 1, 1, 1]), ([40, 300], [3, 9]), ([0, 129], [150, 2])])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 40)])
def test_query_heads_of_a_key_value_head(Hq, Hkv, ctx, new, dtype, D):
    s = Step(ctx, new, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, pad=1, seed=Hq)
    s.map_and_append()
    s.compare()
    s.compare(window=100, softcap=12.0)
    s.close()


@pytest.mark.parametrize("new,Hq,Hkv", [
    ([1] * 20, 16, 1),            # sixteen rows a tile: the second eight are merged, too
    ([3, 2, 1, 3] * 3, 8, 2),     # nine to twelve
    ([1] * 30, 6, 3),
    ([2] * 200, 4, 4),            # many tiles: whole ones
    ([5, 40, 1, 90, 17], 8, 2),   # two tiles, with and without a second stream
])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 128), ("fp16", 64), ("bf16", 80)])
@pytest.mark.parametrize("mask", [{}, dict(window=200, softcap=20.0)])
def test_shared_prefixes_in_every_form(new, Hq, Hkv, dtype, D, mask):
    R, prefix = len(new), 256
    ctx = prefix + np.random.default_rng(R).integers(0, 150, size=R)
    ctx[0] = prefix
    s = Step(ctx, new, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, bt=32, group_start=[0, R // 2, R], prefix=[prefix, prefix - 64], pad=1)
    s.map_and_append()
    s.compare(**mask)
    a, b = s.forward(**mask), s.forward(**mask)
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    s.close()


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("Hkv,D,ctx", [(4, 64, 1500), (2, 96, 1200), (2, 64, 1200)])
@pytest.mark.parametrize("new", [1, 20])
def test_heads_side_by_side_behind_many_keys(Hkv, D, ctx, new, layout):
    """Rows of less than 256 bytes beside other heads': behind more keys than L2 holds they are fetched 64 bytes at
    a time (the first two shapes; the third is behind fewer)."""
    s = Step([ctx, 30, ctx - 77], [new] * 3, Hq=2 * Hkv, Hkv=Hkv, D=D, layout=layout)
    s.map_and_append()
    s.compare()
    s.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("new", [1, 4, 60])
def test_a_query_that_is_not_finite_spoils_its_own_rows_alone(new, bad):
    s = Step([100, 700, 33], [new] * 3, Hq=4, Hkv=2, D=64)
    s.map_and_append()
    clean = s.forward()
    at = new + new // 2  # of the second request
    s.q[at, 1, 5] = bad
    got = s.forward()
    same = np.ones((s.N, s.Hq), dtype=bool)
    same[at, 1] = False
    assert np.array_equal(got[0][same], clean[0][same]) and np.array_equal(got[1][same], clean[1][same])
    assert np.isnan(got[0][at, 1]).all() and np.isnan(got[1][at, 1])
    s.close()


@pytest.mark.parametrize("ctx,new", [([300] * 200, 33), ([300], 60), ([300] * 300, 3), ([3000] * 12, 3), ([3000] * 2, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_near_the_end_of_the_range(ctx, new, D):
    """Values of 3e37, and a key of the second tile whose probability is 2^7 times that of the maximum so far: the
    unscaled sum is past fp32 before it is divided, the result is not.  (One rounding of each probability and one of
    the result, 2^-8 each, and 1e-4 for the fp32 steps.)"""
    R = len(ctx)
    s = Step(ctx, [new] * R, Hq=2, Hkv=1, D=D)
    for c, fill in ((s.kv[0], 0.0), (s.kv[1], 3e37)):
        c.nan_to_num_(0.0).fill_(fill)
    table = s.maps()[0]
    for r in range(R):
        s.kv[0][int(table[r, 200 // s.bt]), 200 % s.bt] = 7 * np.log(2.0) / np.sqrt(D)
    s.q.fill_(1.0)
    s.k.fill_(0.0)
    s.v.fill_(3e37)
    s.map_and_append()
    got, _ = s.forward()
    want, _, absum, _, _ = s.expect()
    assert np.isfinite(want).all() and (np.abs(got - want) <= 2.0 ** -8 * (np.abs(want) + absum) + 1e-4 * absum).all()
    s.close()
