"""Paged attention on the GPU against the float64 oracle (oracle/attn.py): step maps and cache
writes exactly, attention within rounding."""
import numpy as np
import pytest

from attn_helpers import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


LENGTHS = {
    "one": ([0], [1]),
    "one_behind_many": ([300], [1]),
    "decode": ([0, 15, 16, 17, 127, 128, 129, 400], [1] * 8),
    "drafts": ([5, 250, 31], [3, 4, 1]),
    "empty_requests": ([0, 40, 0, 9], [0, 2, 5, 0]),
    "prompt": ([0], [200]),
    "ragged_chunks": ([0, 100, 33, 256], [130, 1, 257, 64]),
}


@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("lengths", sorted(LENGTHS))
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_maps_and_cache_write_are_exact(lengths, bt, layout):
    ctx, new = LENGTHS[lengths]
    R = len(ctx)
    s = Step(ctx, new, Hq=2, Hkv=2, D=24, bt=bt, layout=layout, pad=3, rows=list(np.random.default_rng(bt).permutation(R + 2)[:R]),
             spare_ids=2)
    before = [c.float().cpu().numpy().copy() for c in s.kv]
    s.map_and_append()
    s.pw.pw_attn_check(s.attn)
    table, q_start, kv_len, slot, pos = s.maps()
    for got, want in ((s.table, table), (s.q_start, q_start), (s.kv_len, kv_len), (s.slot, slot), (s.pos, pos)):
        assert np.array_equal(got.cpu().numpy(), want)
    from oracle import attn as oa
    for cache, old, rows in zip(s.kv, before, (s.k, s.v)):
        oa.append(old, rows.float().cpu().numpy(), slot)
        assert np.array_equal(cache.float().cpu().numpy(), old, equal_nan=True)
    s.close()


def test_maps_of_many_requests():
    rng = np.random.default_rng(5)
    ctx, new = rng.integers(0, 90, size=3000), rng.integers(0, 4, size=3000)
    s = Step(ctx, new, Hq=1, Hkv=1, D=8)
    s.map_and_append()
    s.pw.pw_attn_check(s.attn)
    for got, want in zip((s.table, s.q_start, s.kv_len, s.slot, s.pos), s.maps()):
        assert np.array_equal(got.cpu().numpy(), want)
    s.close()


HEADS = [(4, 2, 64, "bf16"), (8, 1, 128, "bf16"), (6, 2, 80, "fp16"), (2, 2, 128, "fp16"), (7, 1, 8, "bf16"),
         (32, 1, 104, "fp16")]


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "-".join(map(str, h)))
@pytest.mark.parametrize("lengths", sorted(LENGTHS))
def test_causal(lengths, heads):
    Hq, Hkv, D, dtype = heads
    s = Step(*LENGTHS[lengths], Hq=Hq, Hkv=Hkv, D=D, dtype=dtype, pad=2)
    s.map_and_append()
    s.compare()
    s.close()


@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_block_sizes_and_layouts(bt, layout):
    s = Step([0, 77, 300], [150, 1, 20], D=128, bt=bt, layout=layout, rows=[4, 0, 2])
    s.map_and_append()
    s.compare()
    s.close()


MASKS = {
    "window_1": dict(window=1),
    "window_100": dict(window=100),
    "cap": dict(softcap=5.0),
    "bias": dict(slopes=True),
    "window_cap_bias": dict(window=150, softcap=20.0, slopes=True),
    "documents": dict(docs=True),
    "two_way_prefix": dict(bidir=True),
    "everything": dict(window=190, softcap=9.0, slopes=True, docs=True, bidir=True),
    "scale": dict(scale=0.5),
    "negative_scale": dict(scale=-0.25),
}


def _mask(s, docs=False, bidir=False, slopes=False, **kw):
    rng = np.random.default_rng(9)
    if docs:
        parts = []
        for c, n in zip(s.ctx, s.new):
            cuts = np.concatenate([[0], np.sort(rng.integers(0, c + n + 1, size=3))])
            p = np.arange(c, c + n)
            parts.append(cuts[np.searchsorted(cuts, p, side="right") - 1])
        kw["doc_start"] = np.concatenate(parts + [np.zeros(s.N - sum(s.new))])
    if bidir:
        kw["bidir_len"] = [int(rng.integers(0, c + n + 40)) for c, n in zip(s.ctx, s.new)]
    if slopes:
        kw["slopes"] = 2.0 ** (-8.0 * np.arange(1, s.Hq + 1) / s.Hq)
    return kw


@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("lengths", ["one", "decode", "drafts", "ragged_chunks"])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("fp16", 128)])
def test_masks(mask, lengths, dtype, D):
    s = Step(*LENGTHS[lengths], D=D, dtype=dtype, pad=1, seed=2)
    s.map_and_append()
    s.compare(**_mask(s, **MASKS[mask]))
    s.close()


@pytest.mark.parametrize("new", [1, 70])
def test_rows_whose_mask_leaves_nothing(new):
    """A document that begins behind the row's own position leaves it no key."""
    s = Step([140, 3, 0], [new, 2, 5], D=64)
    s.map_and_append()
    doc = np.zeros(s.N)
    doc[:new] = np.where(np.arange(new) % 2 == 0, 1000, 0)
    doc[new:] = 1000
    if new == 70:
        doc[:new] = np.sort(doc[:new])
    s.compare(doc_start=doc)
    s.close()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("which", ["k", "v"])
def test_values_behind_the_mask_do_not_reach_a_row(value, dtype, which):
    """One cached token holds infinities or NaN; the rows that do not see it are as without it."""
    s = Step([200], [90], D=64, dtype=dtype)
    s.map_and_append()
    s.torch.cuda.synchronize()
    where = 215  # seen by the rows at 215 .. 290 but not by those before
    page = s.maps()[0][0, where // s.bt]
    s.kv[0 if which == "k" else 1][int(page), where % s.bt] = value
    got, lse = s.forward()
    o, want_lse, absum, xmax, bounds = s.expect()
    free = np.array([hi <= where for _, _, lo, hi in bounds])
    assert free.sum() == 15 and np.isfinite(got[free]).all() and np.isfinite(lse[free]).all()
    tol = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}[dtype] * (np.abs(o) + absum) + 1e-4 * absum + 1e-4
    assert (np.abs(got - o)[free] <= tol[free]).all()
    if which == "v":
        assert not np.isfinite(got[~free]).any()
    s.close()


@pytest.mark.parametrize("new,group_start,prefix", [
    ([1] * 9, [0, 9], 256), ([1] * 9, [0, 4, 9], [128, 16]), ([1] * 9, [0, 1, 2, 9], [64, 0, 272]),
    ([3, 70, 1, 0, 2], [0, 5], 160), ([1] * 40, [0, 40], 1024)])
@pytest.mark.parametrize("mask", ["none", "everything", "window_100"])
def test_shared_prefix(new, group_start, prefix, mask):
    R = len(new)
    lens = [prefix] * (len(group_start) - 1) if np.isscalar(prefix) else prefix
    rng = np.random.default_rng(R)
    ctx = []
    for g in range(len(group_start) - 1):
        ctx += [lens[g] + int(rng.integers(0, 60)) for _ in range(group_start[g], group_start[g + 1])]
    ctx[0] = lens[0]
    s = Step(ctx, new, Hq=4, Hkv=1, D=64, group_start=group_start, prefix=lens, pad=2)
    s.map_and_append()
    s.compare(**_mask(s, **MASKS.get(mask, {})))
    s.close()


@pytest.mark.parametrize("new", [[0, 0, 0], [0, 2, 0]])
def test_shared_prefix_of_requests_without_new_tokens(new):
    s = Step([48, 70, 33], new, Hq=4, Hkv=1, D=64, group_start=[0, 1, 3], prefix=[48, 32], pad=3)
    s.map_and_append()
    s.compare()
    s.close()


def test_long_context_is_split():
    s = Step([20000], [1], Hq=2, Hkv=1, D=64, bt=64)
    s.map_and_append()
    s.compare()
    s.compare(slopes=[0.01, 0.002])
    s.close()


def test_calls_repeat_bit_for_bit_and_follow_new_lengths():
    """The same plan twice gives the same bits; a step of other lengths through the same handle
    gives its own results."""
    s = Step([900, 20, 333], [1, 1, 1], D=128)
    s.map_and_append()
    a, b = s.forward(), s.forward()
    assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])
    s.compare()
    s.compare(window=37)
    s.compare()
    s.close()


@pytest.mark.parametrize("group_start", [None, [0, 3]])
@pytest.mark.parametrize("kw", [dict(), dict(window=40, softcap=30.0), dict(softcap=2.0), dict(slopes=[0.3] * 8)])
def test_bits_do_not_depend_on_unwritten_memory(kw, group_start):
    """Whatever the cache holds behind the written tokens, and whatever ran before: the same bits."""
    ref = None
    for fill in (float("nan"), 0.0, 1e30, -3.0):
        s = Step([80, 80, 80], [13, 1, 50], Hq=8, Hkv=2, D=32, seed=3, group_start=group_start, prefix=80)
        for c in s.kv:
            c[s.torch.isnan(c)] = fill
        s.map_and_append()
        for _ in range(10):
            got = s.forward(**kw)
            ref = ref or got
            assert np.array_equal(got[0], ref[0]) and np.array_equal(got[1], ref[1])
        s.close()


def test_step_in_a_cuda_graph_follows_the_lengths():
    import torch
    s = Step([100, 40], [1, 1], D=64, spare_ids=2)
    s.map_and_append()
    s.compare()
    o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        s.pw.pw_kv_map(s.attn, s.step, s.new_ids, stream=st)
        s.pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v, stream=st)
        s.pw.pw_attn_plan(s.attn, 0, s.step, stream=st)
        s.pw.pw_attn_forward(s.attn, 0, 0, s.q, o, stream=st)
    ctx_dev, new_dev = s.step.refs[:2]
    for ctx, new in (([100, 40], [1, 1]), ([60, 33], [1, 1]), ([99, 0], [2, 0])):
        s.ctx, s.new = ctx, new
        ctx_dev.copy_(torch.tensor(ctx, dtype=torch.int32))
        new_dev.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        want, _, absum, _, where = s.expect()
        n = len(where)
        got = o.float().cpu().numpy()
        assert (np.abs(got[:n] - want) <= 2.0 ** -8 * (np.abs(want) + absum) + 1e-4 * absum).all()
        assert not got[n:].any()
    s.close()


def test_findings_of_the_map_are_reported_once():
    def finding(change, text):
        s = Step([20, 5], [4, 30], D=64)
        s.torch.cuda.synchronize()
        change(s)
        s.pw.pw_kv_map(s.attn, s.step, s.new_ids)
        s.pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v)
        with pytest.raises(s.pw.PwError) as e:
            s.pw.pw_attn_check(s.attn)
        assert e.value.status == s.pw.PW_ERR_STATE and text in str(e.value)
        s.pw.pw_attn_check(s.attn)
        # what was not concerned is still right, what was is -1
        slot = s.slot.cpu().numpy()
        assert ((slot == -1) | (slot >= 0)).all() and (slot < s.n_blocks * s.bt).all()
        # and attention over such a map reads nothing out of range
        o = s.torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
        s.pw.pw_attn_plan(s.attn, 0, s.step)
        s.pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
        s.pw.pw_attn_check(s.attn)
        s.close()

    def few_ids(s):
        s.new_ids = s.new_ids[:-1]

    def foreign_id(s):
        s.new_ids[0] = s.n_blocks

    def negative_length(s):
        s.step.refs[0][1] = -4

    def long_request(s):
        s.step.refs[0][0] = 1 << 20

    def many_tokens(s):
        s.step.refs[1][1] = 31

    finding(few_ids, "fewer new ids")
    finding(foreign_id, "block id")
    finding(negative_length, "length out of range")
    finding(long_request, "length out of range")
    finding(many_tokens, "more new tokens")


@pytest.mark.parametrize("new", [[1, 1, 1], [70, 1, 4]])
@pytest.mark.parametrize("groups", [False, True])
def test_an_expired_device_wait_is_reported_once(new, groups):
    """One arrival withheld and a short limit (2 ms): PW_ERR_TIMEOUT once, then results as before."""
    kw = dict(group_start=[0, 3], prefix=64) if groups else {}
    s = Step([100, 400, 64], new, Hq=4, Hkv=2, D=64, **kw)
    s.map_and_append()
    s.compare()
    s.pw.pw_attn_set_fault(s.attn, 5, 2000)
    s.pw.pw_attn_set_fault(s.attn, 4, 1)
    o = s.torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    s.pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
    with pytest.raises(s.pw.PwError) as e:
        s.pw.pw_attn_check(s.attn)
    assert e.value.status == s.pw.PW_ERR_TIMEOUT
    s.pw.pw_attn_check(s.attn)
    s.pw.pw_attn_set_fault(s.attn, 5, 0)
    s.compare()
    s.compare(window=33)
    with pytest.raises(s.pw.PwError):
        s.pw.pw_attn_set_fault(s.attn, 1, 1)
    s.close()


def test_refusals_of_the_calls():
    import torch
    s = Step([20], [2], D=64)
    pw, bad = s.pw, []

    def refused(status, call, *a, **k):
        with pytest.raises(pw.PwError) as e:
            call(*a, **k)
        assert e.value.status == status, str(e.value)

    o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    refused(pw.PW_ERR_STATE, pw.pw_attn_forward, s.attn, 0, 0, s.q, o)  # no plan yet
    s.map_and_append()
    pw.pw_attn_plan(s.attn, 0, s.step)
    inv = pw.PW_ERR_INVALID
    refused(inv, pw.pw_attn_forward, s.attn, 1, 0, s.q, o)
    refused(inv, pw.pw_attn_forward, s.attn, 0, 1, s.q, o)
    refused(inv, pw.pw_attn_forward, s.attn, 0, 0, s.q, o, scale=float("nan"))
    refused(inv, pw.pw_attn_forward, s.attn, 0, 0, s.q, o, softcap=-1.0)
    flat = torch.empty(s.N * s.Hq * s.D + 8, dtype=s.dt, device="cuda")
    refused(inv, pw.pw_attn_forward, s.attn, 0, 0, s.q, flat[1:1 + o.numel()].view(o.shape))
    refused(inv, pw.pw_attn_plan, s.attn, 0, s.step, window=-1)
    refused(inv, pw.pw_attn_plan, s.attn, 1, s.step)
    refused(inv, pw.pw_attn_append, s.attn, 2, s.step, s.k, s.v)
    with pytest.raises(ValueError):
        pw.pw_attn_forward(s.attn, 0, 0, s.q, torch.empty(s.N, s.D, s.Hq, dtype=s.dt, device="cuda").transpose(1, 2))
    s.step.R = 2
    refused(inv, pw.pw_kv_map, s.attn, s.step, s.new_ids)
    s.step.R, s.step.n_groups = 1, 1
    refused(inv, pw.pw_kv_map, s.attn, s.step, s.new_ids)
    s.step.n_groups = 0
    pw.pw_attn_check(s.attn)
    s.close()
    assert not bad


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 257])
@pytest.mark.parametrize("dtype,D,mask", [("bf16", 128, {}), ("fp16", 64, dict(softcap=6.0)),
                                          ("bf16", 64, dict(window=70)), ("fp16", 128, dict(softcap=3.0, slopes=True))])
def test_row_counts_around_the_tile_sizes(rows, dtype, D, mask):
    """One request with `rows` new tokens (unshared heads: as many rows in a tile) behind a cache, beside
    one with a single token."""
    s = Step([150, 333], [rows, 1], Hq=2, Hkv=2, D=D, dtype=dtype, bt=32, seed=rows, qscale=2.5)
    s.map_and_append()
    s.compare(**_mask(s, **mask))
    s.close()


@pytest.mark.parametrize("new", [1, 2, 30])
def test_many_requests_share_the_sms(new):
    """More pieces than SMs, most of them short, some tiles split."""
    rng = np.random.default_rng(new)
    R = 150 if new < 30 else 40
    s = Step(rng.integers(0, 700, size=R), [new] * R, Hq=8, Hkv=4, D=64, dtype="fp16")
    s.map_and_append()
    s.compare()
    s.compare(window=200, softcap=15.0)
    s.close()


def test_capped_scores_beyond_the_polynomial():
    """Scores of several times the cap: the tanh is at its ends."""
    s = Step([300, 20], [3, 140], D=64, dtype="fp16", qscale=30.0)
    s.map_and_append()
    s.compare(softcap=4.0)
    s.close()


def test_blocks_beyond_32_bit_offsets():
    """Block ids whose elements lie past 2^32 in the cache."""
    import torch

    import any_precision_bit_gb300 as pw
    n_blocks, bt, Hkv, D = 40000, 128, 8, 128
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 25 GB")
    k = torch.empty(n_blocks, bt, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = torch.tensor([[39990, 5, 33000]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(1)
    rows = [torch.randn(300, Hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    q = torch.randn(300, Hkv, D, generator=g).to(torch.bfloat16).cuda()
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    a = pw.pw_attn_create(pw.pw_attn_desc(L=1, n_heads=Hkv, n_kv_heads=Hkv, head_dim=D, dtype=0, n_blocks=n_blocks,
                                          block_tokens=bt, max_requests=1, max_tokens=300, max_shared_tokens=0, n_plans=1,
                                          device=0))
    pw.pw_attn_bind(a, 0, k, v)
    step = pw.pw_make_step(i32(1), i32(1) + 300, table, i32(2), i32(1), torch.zeros(300, dtype=torch.int64, device="cuda"),
                           i32(300), max_new=300)
    ids = table[0].clone()
    table.fill_(-1)
    torch.cuda.synchronize()
    pw.pw_kv_map(a, step, ids)
    pw.pw_attn_append(a, 0, step, *rows)
    pw.pw_attn_plan(a, 0, step)
    o = torch.empty_like(q)
    pw.pw_attn_forward(a, 0, 0, q, o)
    pw.pw_attn_check(a)
    assert torch.equal(torch.cat([k[i] for i in (39990, 5, 33000)])[:300], rows[0])
    x = torch.einsum("thd,jhd->htj", q.double(), rows[0].double()) / D ** 0.5
    x = x.masked_fill(torch.ones(300, 300, dtype=torch.bool, device="cuda").triu(1), -np.inf)
    p = torch.softmax(x, -1)
    want = torch.einsum("htj,jhd->thd", p, rows[1].double())
    size = torch.einsum("htj,jhd->thd", p, rows[1].double().abs())
    assert bool(((o.double() - want).abs() <= 2.0 ** -8 * (want.abs() + size) + 1e-4 * size).all())
    pw.pw_attn_destroy(a)


@pytest.mark.parametrize("new", [1, 3, 300])
@pytest.mark.parametrize("mask", [{}, dict(softcap=40.0), dict(slopes=True)])
def test_small_probabilities_behind_a_large_one(new, mask):
    """A first key that takes nearly all the weight and whose value is zero: the result is what the others'
    probabilities, about 2^-25 of the largest, add up to.  The largest is 2^7 or more before it is rounded to fp16,
    so a probability is off by 2^-11 of itself or 2^-32 of the largest."""
    R = 160 if new < 100 else 12
    s = Step([300] * R, [new] * R, D=64, dtype="fp16", bt=16)
    first = s.torch.as_tensor(s.table0[:, 0].astype(np.int64)).cuda()
    for c, rest, top in ((s.kv[0], 0.0, 2.1875), (s.kv[1], 16.0, 0.0)):
        c.nan_to_num_(0.0).fill_(rest)
        c[first, 0] = top
    s.q.fill_(1.0)  # the first key's score is 64 * 2.1875 / 8 = 17.5, the others' are 0
    s.k.fill_(0.0)
    s.v.fill_(16.0)
    s.map_and_append()
    kw = dict(mask)
    if kw.pop("slopes", None):
        kw["slopes"] = np.full(s.Hq, 2.0 ** -12)
    got, _ = s.forward(**kw)
    o, _, absum, _, where = s.expect(**kw)
    keys = max(hi - lo for _, _, lo, hi in where)
    # (scores are fp32: 17.5 log2 e with an error of 2^-22 or so, far below 2^-11; results below 2^-14 are subnormal)
    tol = 2.0 ** -11 * (np.abs(o) + absum) + 1e-4 * absum + keys * 2.0 ** -32 * 16.0 + 2.0 ** -25
    assert (o[:, :, 0] > 20 * tol[:, :, 0]).all()
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / tol).max())
    s.close()


def test_plan_refuses_more_work_than_it_can_count():
    """Key tiles are counted in 31 bits over all tiles of rows."""
    import torch
    s = Step([20] * 4, [300] * 4, D=64)
    s.map_and_append()
    s.pw.pw_attn_plan(s.attn, 0, s.step)
    stride = s.step.table_stride
    s.step.table_stride = (2 ** 31 - 1) // s.bt  # 2^24 key tiles a row
    s.step.max_new = 1  # a token a tile: 1200 tiles
    with pytest.raises(s.pw.PwError) as e:
        s.pw.pw_attn_plan(s.attn, 0, s.step)
    assert e.value.status == s.pw.PW_ERR_INVALID
    s.step.table_stride, s.step.max_new = stride, 300
    torch.cuda.synchronize()
    s.compare()
    s.close()


def test_refusals_of_tensors_that_do_not_fit():
    """Tensors of another shape, type or device than the handle and the step ask for never reach a kernel."""
    import torch
    s = Step([20, 7], [2, 3], D=64)
    pw = s.pw
    s.map_and_append()
    pw.pw_attn_plan(s.attn, 0, s.step)
    o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    lse = torch.empty(s.N, s.Hq, device="cuda")
    i32 = torch.zeros(s.N, dtype=torch.int32, device="cuda")
    wrong = [
        lambda: pw.pw_attn_append(s.attn, 0, s.step, s.k[:-1], s.v),
        lambda: pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v[:, :1]),
        lambda: pw.pw_attn_append(s.attn, 0, s.step, s.k.float(), s.v),
        lambda: pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v.cpu()),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q[1:], o),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o[..., :32]),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o.float()),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o, lse=lse[:-1]),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o, lse=lse.double()),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o, slopes=lse[0, :-1]),
        lambda: pw.pw_attn_plan(s.attn, 0, s.step, doc_start=i32[1:]),
        lambda: pw.pw_attn_plan(s.attn, 0, s.step, bidir_len=i32[:1]),
        lambda: pw.pw_attn_bind(s.attn, 0, s.kv[0][1:], s.kv[1][1:]),
        lambda: pw.pw_attn_bind(s.attn, 0, s.kv[0].float(), s.kv[1].float()),
        lambda: pw.pw_make_step(i32[:2], i32[:1], s.table, s.q_start, s.kv_len, s.slot, s.pos, max_new=3),
        lambda: pw.pw_make_step(i32[:2], i32[:2], s.table, s.q_start[:-1], s.kv_len, s.slot, s.pos, max_new=3),
        lambda: pw.pw_make_step(i32[:2], i32[:2], s.table, s.q_start, s.kv_len, s.slot.int(), s.pos, max_new=3),
        lambda: pw.pw_make_step(i32[:2], i32[:2], s.table.long(), s.q_start, s.kv_len, s.slot, s.pos, max_new=3),
        lambda: pw.pw_make_step(i32[:2].cpu(), i32[:2], s.table, s.q_start, s.kv_len, s.slot, s.pos, max_new=3),
    ]
    for call in wrong:
        with pytest.raises(ValueError):
            call()
    s.compare()
    s.close()
