"""Attention of drafted trees against the float64 oracle: every row over the keys before its tree and its ancestors."""
import numpy as np
import pytest

from tree_helpers import UNIT, TreeStep, chain, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


def run(ctx, new, trees, check=None, **kw):
    masks = {k: kw.pop(k) for k in ("window", "softcap", "slopes", "scale") if k in kw}
    s = TreeStep(ctx, new, trees, **kw)
    try:
        s.map_and_append()
        s.compare(**masks)
    finally:
        s.close()


@pytest.mark.parametrize("n", [1, 2, 3, 7, 8, 9, 31, 32, 33, 64, 65, 127, 129, 200, 256])
@pytest.mark.parametrize("ctx", [0, 97, 127, 128, 130])
def test_sizes(n, ctx):
    run([ctx], [n], [random_tree(n, n + ctx)], Hq=2, Hkv=1, D=64, seed=n)


@pytest.mark.parametrize("tree", [[-1] * 20, chain(20), [-1] + [0] * 19, [-1, 0, 0, 1, 1, 2, 2, 3, 3, 4, 4, 5, 5, 6, 6],
                                  chain(256), [-1, 0] * 10], ids=["roots", "chain", "star", "binary", "long chain", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_shapes_of_trees(tree, dtype):
    run([45], [len(tree)], [tree], Hq=4, Hkv=2, D=32, dtype=dtype)


@pytest.mark.parametrize("heads", [(4, 4), (4, 1), (6, 2), (16, 1), (40, 1), (3, 3)], ids=str)
@pytest.mark.parametrize("D", [8, 72, 96, 128])
def test_heads(heads, D):
    run([60, 0], [5, 3], [random_tree(5, 1), random_tree(3, 2)], Hq=heads[0], Hkv=heads[1], D=D, bt=32)


@pytest.mark.parametrize("bt,layout", [(16, "hnd"), (64, "nhd"), (128, "nhd")])
def test_layouts(bt, layout):
    run([200, 77], [40, 3], [random_tree(40, 5), random_tree(3, 6)], bt=bt, layout=layout)


# some nodes are in the cache; all are, and none is new; a request without a tree; one whose tree follows new tokens
MIXED = dict(ctx=[50, 131, 90, 0, 7], new=[6, 0, 17, 140, 30],
             trees=[random_tree(20, 3), random_tree(12, 4), [], random_tree(9, 5), random_tree(30, 6, back=4)])


@pytest.mark.parametrize("kind", [{}, dict(window=1), dict(window=2), dict(window=5), dict(window=60), dict(softcap=2.0),
                                  dict(slopes=[0.5, 0.25, 0.1, 3.0]), dict(slopes=[1.0, 0.2, 0.3, 0.0], softcap=3.0, window=9),
                                  dict(scale=-0.2), dict(scale=0.0), dict(softcap=1e-3), dict(slopes=[-0.01, 40.0, 0, 1])], ids=str)
@pytest.mark.parametrize("form", [dict(), dict(pad=5), dict(rows=[4, 1, 0, 6, 2], dtype="fp16")], ids=str)
def test_masks(kind, form):
    run(**MIXED, **kind, **form)


# few rows: the form for at most 16
@pytest.mark.parametrize("kind", [{}, dict(window=2), dict(window=40), dict(softcap=2.0), dict(slopes=[0.5, 0.25, 0.1, 3.0]),
                                  dict(slopes=[1.0, 0.2, 0.3, 0.0], softcap=3.0, window=3), dict(scale=-0.2)], ids=str)
@pytest.mark.parametrize("Hkv,new", [(1, 3), (1, 4), (2, 8), (4, 16), (4, 9)])
def test_few_rows(kind, Hkv, new):
    ctx = [126, 30, 252, 3]
    trees = [random_tree(new, 1), random_tree(new + 25, 2), [], chain(new)]
    run(ctx, [new] * 4, trees, Hkv=Hkv, **kind)


@pytest.mark.parametrize("n,kind", [(4, {}), (40, {}), (40, dict(slopes=[1e-4, 0.5])), (200, dict(softcap=4.0)), (3, dict(window=30000))])
def test_long_contexts_split_among_sms(n, kind):
    run([40001], [n], [random_tree(n, 7)], Hq=2, Hkv=1, D=64, bt=128, **kind)


@pytest.mark.parametrize("kind", [{}, dict(window=70), dict(slopes=[0.5, 0.25, 0.1, 3.0])], ids=str)
@pytest.mark.parametrize("n", [2, 19])
def test_behind_shared_prefixes(n, kind):
    ctx, R = [64 + 20, 64 + 1, 64, 128 + 30, 128], 5
    run(ctx, [n] * R, [random_tree(n + (3 if r == 0 else 0), r) for r in range(R)], group_start=[0, 3, 5], prefix=[64, 128], **kind)


@pytest.mark.parametrize("kind", [{}, dict(window=9), dict(softcap=3.0), dict(slopes=[0.5, 0.25, 0.1, 3.0])], ids=str)
@pytest.mark.parametrize("n,held", [(2, 5), (4, 90), (19, 30), (40, 60)])
def test_trees_that_begin_within_a_shared_prefix(n, held, kind):
    """Nodes of earlier steps, in blocks that the requests share."""
    ctx = [64 + 2, 64 + 1, 64, 128 + 10, 128]
    trees = [random_tree(n + min(held, c), r, back=20) for r, c in enumerate(ctx)]
    run(ctx, [n] * 5, trees, group_start=[0, 3, 5], prefix=[64, 128], **kind)


def test_many_requests():
    rng = np.random.default_rng(0)
    R = 150
    nodes = rng.integers(0, 12, R)
    held = np.minimum(rng.integers(0, 4, R), nodes)
    new = np.where(nodes == 0, 1, nodes - held)
    ctx = rng.integers(0, 90, R) + held
    run(ctx.tolist(), new.tolist(), [random_tree(int(n), r) for r, n in enumerate(nodes)], Hq=4, Hkv=1, D=32)


@pytest.mark.parametrize("n,ctx", [(3, 300), (40, 300), (40, 20000), (3, 20000)])
@pytest.mark.parametrize("kind", [{}, dict(softcap=3.0, slopes=[0.1, 0.2])], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_a_row_does_not_see_does_not_reach_it(n, ctx, kind, value):
    # node 0 is nobody's parent: its key and value reach its own row alone
    tree = [-1, -1] + [int(p) for p in np.random.default_rng(1).integers(1, np.arange(2, n))]
    s = TreeStep([ctx], [n], [tree], Hq=2, Hkv=1, D=64, bt=64)
    try:
        s.map_and_append()
        slot = int(s.slot[0])
        for c in s.kv:
            c[slot // s.bt, slot % s.bt, 0, 5] = value
        got, lse = s.forward(**kind)
        o, want_lse, absum, _, where = s.expect(**kind)
        s.near(got[1:], o[1:], absum[1:], ctx + n)
        assert np.abs(lse[1:] - want_lse[1:]).max() < 1e-3 and not np.isfinite(got[0, :, 5]).any()
    finally:
        s.close()


@pytest.mark.parametrize("n,ctx", [(3, 300), (40, 300), (40, 20000)])
def test_an_infinite_value_of_an_ancestor_reaches_its_descendants(n, ctx):
    tree = [-1] + [int(p) for p in np.random.default_rng(2).integers(-1, np.arange(1, n))]
    s = TreeStep([ctx], [n], [tree], Hq=2, Hkv=1, D=64, bt=64)
    try:
        s.map_and_append()
        slot = int(s.slot[1])
        s.kv[1][slot // s.bt, slot % s.bt, 0, 3] = float("inf")
        got, _ = s.forward()
        seen = np.array([ctx + 1 in w[2] for w in s.expect()[4]])
        assert np.isposinf(got[seen][:, :, 3]).all() and np.isfinite(got[~seen]).all()
        assert np.isfinite(np.delete(got, 3, axis=2)).all()
    finally:
        s.close()


def test_a_chain_and_no_tree_are_what_a_plain_plan_is():
    """The plain plan's formula with Step.compare's tolerances, and its positions."""
    ctx, new = [70, 5, 300], [20, 33, 1]
    for trees in ([chain(n) for n in new], [[], [], []], [chain(25), [], chain(1)]):
        s = TreeStep(ctx, new, trees)
        try:
            s.map_and_append()
            got, lse = s.forward(window=50)
            o, want_lse, absum, xmax, _ = super(TreeStep, s).expect(window=50)
            s.near(got, o, absum, 50)
            assert (np.abs(lse - want_lse) <= 2.0 ** -23 * (s.D + 16) * (4.0 + xmax)).all()
            assert s.tree_pos.tolist() == s.pos.tolist()
        finally:
            s.close()


def test_findings_are_reported():
    ctx, new = [20, 20, 3, 40], [5, 5, 4, 6]
    good = [random_tree(5, 1), random_tree(5, 2), [], random_tree(6, 3)]
    s = TreeStep(ctx, new, good)
    pw = s.pw
    try:
        s.map_and_append()
        s.compare()
        for r, node, parent in ((1, 2, 2), (1, 0, 0), (3, 4, -2), (3, 1, 77)):
            s.set_trees(good)
            s.parent[r, node] = parent
            s.trees[r] = [-1 if i == node else p for i, p in enumerate(good[r])]
            got, _ = s.forward(check=False)
            with pytest.raises(pw.PwError) as e:
                pw.pw_attn_check(s.attn)
            assert e.value.status == pw.PW_ERR_STATE and "tree" in str(e.value)
            o, _, absum, _, _ = s.expect()
            s.near(got, o, absum, 64)
        for r, length in ((0, -1), (0, 257), (2, 8), (1, 7), (3, 1 << 30)):  # (7: more than parent has columns)
            s.set_trees(good)
            s.tree_len[r] = length
            s.trees[r] = []
            got, _ = s.forward(check=False)
            with pytest.raises(pw.PwError):
                pw.pw_attn_check(s.attn)
            o, _, absum, _, _ = s.expect()
            s.near(got, o, absum, 64)
        s.set_trees(good)
        s.compare()
    finally:
        s.close()


def test_refusals():
    s = TreeStep([20], [5], [random_tree(5, 1)], n_plans=2)
    pw, t = s.pw, s.torch
    try:
        step, tl, par = s.step, s.tree_len, s.parent
        plan = lambda **kw: pw.pw_attn_plan_tree(**{**dict(attn=s.attn, plan=0, step=step, tree_len=tl, parent=par), **kw})  # noqa: E731
        for change in (dict(plan=2), dict(plan=-1), dict(window=-1)):
            with pytest.raises(pw.PwError) as e:
                plan(**change)
            assert e.value.status == pw.PW_ERR_INVALID
        for change in (dict(tree_len=tl.long()), dict(tree_len=tl.cpu()), dict(parent=par.cpu()), dict(parent=par.T.expand(5, 4)),
                       dict(pos=s.pos[:3]), dict(tree_len=tl[:0])):
            with pytest.raises((ValueError, TypeError)):
                plan(**change)
        short = pw.pw_attn_create(pw.pw_attn_desc(L=1, n_heads=4, n_kv_heads=2, head_dim=64, dtype=0, n_blocks=s.n_blocks,
                                                  block_tokens=16, max_requests=1, max_tokens=5, n_plans=1, device=0,
                                                  max_tree_tokens=4))
        try:
            with pytest.raises(pw.PwError) as e:
                plan(attn=short)
            assert e.value.status == pw.PW_ERR_INVALID and "max_tree_tokens" in str(e.value)
        finally:
            pw.pw_attn_destroy(short)
        s.map_and_append()
        s.compare()
    finally:
        s.close()


def test_captured_steps_follow_new_trees():
    """Plan and forward in one graph, replayed with other lengths and trees; a forward alone, behind plans of either call."""
    import torch
    s = TreeStep([100, 40, 7], [6, 6, 6], [random_tree(6, 1), random_tree(6, 2), random_tree(6, 3)], Hkv=1)
    pw = s.pw
    try:
        s.map_and_append()
        o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
        stream = torch.cuda.Stream()

        def both():
            s.plan(window=30, stream=stream)
            pw.pw_attn_forward(s.attn, 0, 0, s.q, o, stream=stream)
        stream.wait_stream(torch.cuda.current_stream())
        both()
        torch.cuda.synchronize()
        graph, alone = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            both()
        with torch.cuda.graph(alone, stream=stream):
            pw.pw_attn_forward(s.attn, 0, 0, s.q, o, stream=stream)

        def fits(window):
            torch.cuda.synchronize()
            pw.pw_attn_check(s.attn)
            want, _, absum, _, _ = s.expect(window=window)
            s.near(o.float().cpu().numpy(), want, absum, 128)
        for k in range(3):
            s.set_trees([random_tree(6, 10 + k), random_tree(6, 20 + k), random_tree(6, 30 + k)])
            o.fill_(7.0)
            torch.cuda.synchronize()
            graph.replay()
            fits(30)
        s.set_trees([random_tree(6, 4), random_tree(6, 5), random_tree(6, 6)])
        torch.cuda.synchronize()
        s.plan(window=3)
        torch.cuda.synchronize()
        alone.replay()
        fits(3)
        pw.pw_attn_plan(s.attn, 0, s.step)  # not the call that the forward was captured with
        torch.cuda.synchronize()
        o.fill_(7.0)
        torch.cuda.synchronize()
        alone.replay()
        with pytest.raises(pw.PwError) as e:
            pw.pw_attn_check(s.attn)
        assert e.value.status == pw.PW_ERR_STATE and bool((o == 7).all())
    finally:
        s.close()


@pytest.mark.parametrize("ctx", [0, 120, 130, 250, 260, 390, 1000, 1100])
@pytest.mark.parametrize("kind", [{}, dict(window=140), dict(softcap=3.0), dict(slopes=[0.5, 0.25, 0.1, 3.0])], ids=str)
@pytest.mark.parametrize("D", [64, 128])
def test_one_tile_of_rows_behind_several_of_keys(ctx, kind, D):
    """Odd and even numbers of key tiles, of which two streams take turns; beside rows of two tiles."""
    run([ctx, ctx + 60, ctx // 2], [24, 40, 17], [random_tree(24, ctx), random_tree(40, ctx + 1), random_tree(20, ctx + 2)][:3],
        Hq=8, Hkv=2, D=D, **{**kind, **({"slopes": kind["slopes"] * 2} if "slopes" in kind else {})}) if ctx > 5 else \
        run([ctx], [24], [random_tree(24, ctx)], D=D, **kind)


@pytest.mark.parametrize("n", [3, 24, 70])
def test_an_expired_wait_is_reported_and_the_handle_usable(n):
    s = TreeStep([100, 400, 64], [n] * 3, [random_tree(n, r) for r in range(3)])
    pw = s.pw
    try:
        s.map_and_append()
        s.compare()
        pw.pw_attn_set_fault(s.attn, 5, 2000)
        pw.pw_attn_set_fault(s.attn, 4, 1)
        o = s.torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
        pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
        with pytest.raises(pw.PwError) as e:
            pw.pw_attn_check(s.attn)
        assert e.value.status == pw.PW_ERR_TIMEOUT
        pw.pw_attn_check(s.attn)
        pw.pw_attn_set_fault(s.attn, 5, 0)
        s.compare()
    finally:
        s.close()


def test_a_captured_forward_does_not_fit_a_plan_that_divides_otherwise():
    """Tiles of as many tokens, but with key tiles that weigh otherwise since a request may bring more."""
    import torch
    s = TreeStep([700, 300], [20, 12], [random_tree(20, 1), random_tree(12, 2)], Hq=4, Hkv=1)
    pw = s.pw
    try:
        s.map_and_append()
        o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
        ctx, new, table, q_start, kv_len, slot, pos = s.step.refs[:7]
        wide, narrow = (pw.pw_make_step(ctx, new, table, q_start, kv_len, slot, pos, max_new=n) for n in (64, 32))

        def plan(step):
            pw.pw_attn_plan_tree(s.attn, 0, step, s.tree_len, s.parent, pos=s.tree_pos)
            torch.cuda.synchronize()
        for first, second in ((wide, narrow), (narrow, wide)):
            plan(first)
            pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
            pw.pw_attn_check(s.attn)
            want, _, absum, _, _ = s.expect()
            s.near(o.float().cpu().numpy(), want, absum, 720)
            graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
            with torch.cuda.graph(graph, stream=stream):
                pw.pw_attn_forward(s.attn, 0, 0, s.q, o, stream=stream)
            plan(second)
            o.fill_(7.0)
            torch.cuda.synchronize()
            graph.replay()
            with pytest.raises(pw.PwError) as e:
                pw.pw_attn_check(s.attn)
            assert e.value.status == pw.PW_ERR_STATE and bool((o == 7).all())
    finally:
        s.close()


@pytest.mark.parametrize("n", [3, 24, 40])
@pytest.mark.parametrize("heads", [(2, 1), (8, 2)], ids=str)
def test_short_steps_behind_long_ones_in_one_handle(n, heads):
    """What earlier steps left in the workspace has no say."""
    s = TreeStep([5000], [n], [random_tree(n, 1)], Hq=heads[0], Hkv=heads[1], bt=16, spare_ids=4)
    try:
        for ctx in (5000, 120, 4000, 130, 250, 700, 1500, 20, 0, 380):
            s.ctx = [ctx]
            s.step.refs[0].fill_(ctx)
            s.table.copy_(s.torch.as_tensor(s.table0))  # without the block that the step before opened
            s.map_and_append()
            s.compare()
    finally:
        s.close()


def test_results_repeat_bit_by_bit():
    s = TreeStep([3000, 500, 9000], [64, 13, 40], [random_tree(64, 1), random_tree(13, 2), random_tree(40, 3)], Hq=8, Hkv=2, D=128)
    try:
        s.map_and_append()
        first = s.forward()
        for _ in range(5):
            again = s.forward()
            assert np.array_equal(first[0], again[0]) and np.array_equal(first[1], again[1])
    finally:
        s.close()
