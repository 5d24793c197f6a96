"""Infinities and NaN in written values: rows that do not see them are as without them, rows that do are what
the formula gives, in every form of the kernels (whole tiles, split ones added up by the last CTA or by the
summing kernel, shared prefixes and what lies behind them)."""
import numpy as np
import pytest

from attn_helpers import UNIT, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


def _many(R, lo, hi, new, seed=3):
    return np.random.default_rng(seed).integers(lo, hi, size=R), [new] * R


# name: (ctx, new, keywords of Step, position of the bad key of a request from its ctx, keywords of forward)
SHAPES = {
    # two tiles: whole ones and some cut by an SM's share; a summing kernel for one request's
    "two_whole": (*_many(200, 100, 300, 33), dict(Hq=2, Hkv=1, D=80), 9, {}),
    "two_whole_long": (*_many(200, 3900, 4000, 33), dict(Hq=2, Hkv=1, D=8), 9, {}),
    "two_whole_one_stream": (*_many(200, 100, 300, 17), dict(Hq=2, Hkv=2, D=128), 9, {}),
    "two_join": ([200], [90], dict(Hq=4, Hkv=2, D=128), 15, {}),
    "two_join_long": ([6000, 30], [90, 2], dict(Hq=4, Hkv=2, D=80), 15, {}),
    # few rows: whole, split and added up by the last CTA, split and summed by a kernel
    "few_whole": (*_many(400, 100, 300, 3), dict(Hq=4, Hkv=1, D=64), 1, {}),
    "few_whole_sixteen": (*_many(400, 100, 300, 4), dict(Hq=8, Hkv=2, D=128), 2, {}),
    "few_split": (*_many(12, 3900, 4000, 4), dict(Hq=2, Hkv=1, D=80), 2, {}),
    "few_split_one_row": (*_many(12, 3900, 4000, 1), dict(Hq=2, Hkv=2, D=64), -20, {"window": 64}),
    "few_join": (*_many(2, 3900, 4000, 4), dict(Hq=4, Hkv=1, D=128), 2, {}),
    "cap_bias": (*_many(200, 100, 300, 33), dict(Hq=2, Hkv=1, D=64), 9, dict(softcap=9.0, slopes=[0.125, 0.01])),
}


def bad_at(s, where, value):
    """The value rows of position where[r] of each request r (None: of none)."""
    table = s.maps()[0]
    for r, w in enumerate(where):
        if w is not None:
            row = r if s.rows is None else s.rows[r]
            s.kv[1][int(table[row, w // s.bt]), w % s.bt] = value


def check(s, where, value, kw):
    got, lse = s.forward(**kw)
    again = s.forward(**kw)
    assert np.array_equal(got, again[0], equal_nan=True) and np.array_equal(lse, again[1], equal_nan=True)
    o, want_lse, absum, xmax, bounds = s.expect(**kw)
    n = len(bounds)
    sees = np.array([where[r] is not None and lo <= where[r] < hi for r, _, lo, hi in bounds])
    assert sees.any() and not sees.all()
    keys = max(hi - lo for _, _, lo, hi in bounds)
    v = s.kv[1].float()
    vmax = float(v[s.torch.isfinite(v)].abs().max())
    free = ~sees
    tol = UNIT[s.dtype] * (np.abs(o[free]) + absum[free]) + 1e-4 * absum[free] + keys * 2.0 ** -25 * vmax
    assert (np.abs(got[:n][free] - o[free]) <= tol).all()
    if np.isnan(value):
        assert np.isnan(got[:n][sees]).all()
    else:
        assert (got[:n][sees] == value).all()
    some = ~np.isneginf(want_lse)
    assert (np.abs(lse[:n] - want_lse)[some] <= (2.0 ** -23 * (s.D + 16) * (4.0 + xmax))[some]).all()
    assert np.isneginf(lse[:n][~some]).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", sorted(SHAPES))
def test_a_bad_value_that_some_rows_see(shape, dtype, value):
    ctx, new, kw, behind, fwd = SHAPES[shape]
    s = Step(ctx, new, dtype=dtype, **kw)
    s.map_and_append()
    clean = s.forward(**fwd)
    s.torch.cuda.synchronize()
    # in every third request (its rows are the last ones' neighbours in tiles, pieces and warps)
    where = [int(c) + behind if r % 3 == 0 else None for r, c in enumerate(s.ctx)]
    if shape == "few_split_one_row":  # behind the window of every second of them
        where = [w if w is None or r % 2 else w - 60 for r, w in enumerate(where)]
    table = s.maps()[0]
    kept = [None if w is None else s.kv[1][int(table[r, w // s.bt]), w % s.bt].clone() for r, w in enumerate(where)]
    bad_at(s, where, value)
    check(s, where, value, fwd)
    # and nothing of it is left in the next call
    for r, w in enumerate(where):
        if w is not None:
            s.kv[1][int(table[r, w // s.bt]), w % s.bt] = kept[r]
    after = s.forward(**fwd)
    assert np.array_equal(clean[0], after[0]) and np.array_equal(clean[1], after[1])
    s.close()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp16", 128)])
@pytest.mark.parametrize("place", ["prefix", "tail"])
@pytest.mark.parametrize("new,Hq,Hkv", [([3] * 9, 4, 1), ([1] * 40, 8, 2), ([4] * 30, 8, 2), ([3, 70, 1, 20, 66], 4, 2)])
def test_a_bad_value_of_a_shared_prefix_or_behind_it(new, Hq, Hkv, place, dtype, D, value):
    R, prefix = len(new), 512
    ctx = prefix + np.random.default_rng(R).integers(10, 200, size=R)
    ctx[0] = prefix + 150
    s = Step(ctx, new, Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, group_start=[0, R], prefix=prefix)
    s.map_and_append()
    if place == "prefix":  # a window hides it from the later rows
        bad_at(s, [460] + [None] * (R - 1), value)
        where, kw = [460] * R, dict(window=150)
    else:
        where = [int(c) + n - 1 if r % 3 == 0 else None for r, (c, n) in enumerate(zip(s.ctx, s.new))]
        bad_at(s, where, value)
        kw = {}
    check(s, where, value, kw)
    s.close()


SHAPES_OF_WAITS = {n: SHAPES[n] for n in ("two_whole_long", "few_split", "few_whole", "two_join_long")}
SHAPES_OF_WAITS["few_long"] = (*_many(12, 30000, 31000, 4), dict(Hq=2, Hkv=1, D=8), 2, {})
SHAPES_OF_WAITS["few_whole_long"] = (*_many(400, 900, 1000, 4), dict(Hq=4, Hkv=1, D=8), 2, {})


@pytest.mark.parametrize("shape", sorted(SHAPES_OF_WAITS))
def test_the_waits_of_a_call_do_not_depend_on_what_the_values_hold(shape):
    """Bounded waits of 3 ms, behind which the whole call ends where all values are finite: they do not
    expire either where rows have to be computed again, which takes longer."""
    ctx, new, kw, behind, fwd = SHAPES_OF_WAITS[shape]
    s = Step(ctx, new, **kw)
    s.map_and_append()
    s.pw.pw_attn_set_fault(s.attn, 5, 3000)
    s.forward(**fwd)
    where = [max(int(c) - 50, 0) for c in s.ctx]  # seen by all rows
    bad_at(s, where, float("inf"))
    got, _ = s.forward(**fwd)
    assert (got == np.inf).all()
    s.close()


@pytest.mark.parametrize("new", [9, 17, 32])
@pytest.mark.parametrize("ctx", [3, 70, 250])
@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0)])
def test_unwritten_values_beside_quarters_of_a_tile_without_rows(ctx, new, kw):
    """Tiles of 18 to 64 rows: half or more of the warps that clear the values behind the last key have no rows of
    their own.  The same bits whatever lies there."""
    ref = None
    for fill in (0.0, float("nan"), float("inf"), -2.0):
        s = Step([ctx] * 40, [new] * 40, Hq=4, Hkv=2, D=128, seed=5)
        for c in s.kv:
            c[s.torch.isnan(c)] = fill
        s.map_and_append()
        for _ in range(5):
            got = s.forward(**kw)
            ref = ref or got
            assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
        if fill == 0.0:
            s.compare(**kw)
        s.close()


@pytest.mark.parametrize("new,R", [(1, 40), (20, 10)])
def test_the_waits_behind_a_shared_prefix_do_not_depend_on_what_its_values_hold(new, R):
    """The kernel behind the prefix begins while that one's results are added up, and its waits of 3 ms with it; rows
    that are computed again there take longer."""
    s = Step([16384 + 10] * R, [new] * R, Hq=64, Hkv=64, D=8, bt=128, group_start=[0, R], prefix=16384)
    s.map_and_append()
    s.pw.pw_attn_set_fault(s.attn, 5, 3000)
    s.forward()
    bad_at(s, [100] + [None] * (R - 1), float("inf"))
    got, _ = s.forward()
    assert (got == np.inf).all()
    s.close()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("prefix,per", [(256, 4), (1024, 2)])
def test_a_bad_value_in_some_of_many_shared_prefixes(prefix, per, value):
    """More tiles of prefixes than SMs, so that many of them are whole."""
    groups = 100
    R = groups * per
    ctx = prefix + np.random.default_rng(4).integers(0, 120, size=R)
    s = Step(ctx, [1 + r % 2 for r in range(R)], Hq=4, Hkv=2, D=64, bt=32, group_start=list(range(0, R + 1, per)), prefix=prefix)
    s.map_and_append()
    at = prefix - 30
    bad_at(s, [at if r % (3 * per) == 0 else None for r in range(R)], value)
    where = [at if r // per % 3 == 0 else None for r in range(R)]
    check(s, where, value, dict(window=100))
    s.close()
