"""A captured forward, replayed after its plan was laid out again: results of the new lengths and masks, or an
error where the launch does not fit the plan any more."""
import numpy as np
import pytest

from attn_helpers import UNIT, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


class Captured:
    """A step of three requests whose forward alone is in a graph."""

    def __init__(self, new=(4, 4, 4), groups=False, **kw):
        import torch
        self.torch = torch
        if groups:
            kw.update(group_start=[0, 3], prefix=64)
        self.s = s = Step([100, 400, 70], list(new), Hq=4, Hkv=1, D=64, **kw)
        self.pw = s.pw
        s.map_and_append()
        self.o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
        self.stream = torch.cuda.Stream()
        self.pw.pw_attn_plan(s.attn, 0, s.step)
        self.replay_alone()
        self.graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(self.graph, stream=self.stream):
            self.pw.pw_attn_forward(s.attn, 0, 0, s.q, self.o, stream=self.stream)
        self.fits()

    def replay_alone(self):  # the form's first launch is not a captured one
        self.pw.pw_attn_forward(self.s.attn, 0, 0, self.s.q, self.o)
        self.torch.cuda.synchronize()

    def replay(self):
        self.torch.cuda.synchronize()
        self.o.fill_(7.0)
        self.torch.cuda.synchronize()
        self.graph.replay()
        self.torch.cuda.synchronize()

    def fits(self, **kw):
        s = self.s
        self.replay()
        self.pw.pw_attn_check(s.attn)
        want, _, absum, _, where = s.expect(**kw)
        got, n = self.o.float().cpu().numpy(), len(where)
        assert (np.abs(got[:n] - want) <= UNIT[s.dtype] * (np.abs(want) + absum) + 1e-4 * absum).all()
        assert not got[n:].any()

    def does_not_fit(self):
        self.replay()
        with pytest.raises(self.pw.PwError) as e:
            self.pw.pw_attn_check(self.s.attn)
        assert e.value.status == self.pw.PW_ERR_STATE and "plan" in str(e.value)
        self.pw.pw_attn_check(self.s.attn)
        assert bool((self.o == 7.0).all())


@pytest.mark.parametrize("groups", [False, True])
@pytest.mark.parametrize("new", [(4, 4, 4), (1, 1, 1), (70, 3, 40)])
def test_same_shape_other_lengths_and_masks(new, groups):
    c = Captured(new, groups, spare_ids=2)
    s = c.s
    c.pw.pw_attn_plan(s.attn, 0, s.step, window=30)
    c.fits(window=30)
    # fewer tokens in the cache: the maps made again, the plan too
    ctx = [64, 320, 66]
    s.ctx = ctx
    s.step.refs[0].copy_(c.torch.tensor(ctx, dtype=c.torch.int32))
    s.new_ids.copy_(c.torch.as_tensor(s.ids))
    c.torch.cuda.synchronize()
    # (the table's blocks of the old contexts head the row; blocks that the new tokens open are granted again)
    s.table.copy_(c.torch.as_tensor(s.table0))
    need = sum(-(-(a + n) // s.bt) + (-a // s.bt) for a, n in zip(ctx, s.new))
    assert need <= len(s.ids)
    c.pw.pw_kv_map(s.attn, s.step, s.new_ids)
    c.pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v)
    c.pw.pw_attn_plan(s.attn, 0, s.step)
    c.fits()
    s.close()


@pytest.mark.parametrize("groups", [False, True])
@pytest.mark.parametrize("was,then", [(4, 1), (1, 4), (4, 5), (4, 30), (30, 4), (70, 4), (4, 70), (300, 1), (70, 300)])
def test_other_tile_sizes_are_reported(was, then, groups):
    c = Captured((1, 1, 1) if was == 1 else (4, 3, 4) if was < 60 else (70, 3, 40), groups)
    s = c.s
    kept = s.step.max_new
    s.step.max_new = was
    c.pw.pw_attn_plan(s.attn, 0, s.step)
    graph, c.graph = c.graph, c.torch.cuda.CUDAGraph()
    c.replay_alone()
    with c.torch.cuda.graph(c.graph, stream=c.stream):
        c.pw.pw_attn_forward(s.attn, 0, 0, s.q, c.o, stream=c.stream)
    c.fits()
    s.step.max_new = then
    c.pw.pw_attn_plan(s.attn, 0, s.step)
    if min(was, 32) == min(then, 32):  # tiles of 128 rows either way
        c.fits()
    else:
        c.does_not_fit()
    s.step.max_new = was
    c.pw.pw_attn_plan(s.attn, 0, s.step)
    c.fits()
    s.step.max_new = kept
    s.compare()
    del graph
    s.close()


@pytest.mark.parametrize("groups", [False, True])
def test_another_step_in_the_plan_is_reported(groups):
    c = Captured((4, 4, 4), groups)
    s, t = c.s, c.torch
    kw = dict(ctx_len=s.step.refs[0], new_len=s.step.refs[1], table=s.table, q_start=s.q_start, kv_len=s.kv_len, slot=s.slot,
              pos=s.pos, max_new=4, groups=s.groups, shared_len=s.shared)
    wide = t.full((3, s.table.shape[1] + 5), -1, dtype=t.int32, device="cuda")
    wide[:, :s.table.shape[1]] = s.table
    others = [dict(table=s.table.clone()), dict(table=wide),
              dict(slot=s.slot[:11].clone(), pos=s.pos[:11].clone())]
    others.append(dict(groups=None, shared_len=None) if groups else {})
    for change in others:
        if not change:
            continue
        step = c.pw.pw_make_step(**{**kw, **change})
        t.cuda.synchronize()
        c.pw.pw_attn_plan(s.attn, 0, step)
        c.does_not_fit()
        c.pw.pw_attn_plan(s.attn, 0, s.step)
        c.fits()
    s.close()


def test_groups_that_come_later_are_reported():
    import torch
    s = Step([100, 400, 70], [4, 4, 4], Hq=4, Hkv=1, D=64, group_start=[0, 3], prefix=64)
    s.map_and_append()
    pw = s.pw
    alone = pw.pw_make_step(s.step.refs[0], s.step.refs[1], s.table, s.q_start, s.kv_len, s.slot, s.pos, max_new=4)
    o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    pw.pw_attn_plan(s.attn, 0, alone)
    pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        pw.pw_attn_forward(s.attn, 0, 0, s.q, o, stream=stream)
    pw.pw_attn_plan(s.attn, 0, s.step)
    o.fill_(7.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    with pytest.raises(pw.PwError) as e:
        pw.pw_attn_check(s.attn)
    assert e.value.status == pw.PW_ERR_STATE and bool((o == 7.0).all())
    s.close()


def test_a_captured_plan_that_was_never_replayed_is_reported():
    import torch
    s = Step([100, 400, 70], [4, 4, 4], Hq=4, Hkv=1, D=64)
    s.map_and_append()
    pw, stream, graph = s.pw, torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        pw.pw_attn_plan(s.attn, 0, s.step, stream=stream)
    o = torch.full((s.N, s.Hq, s.D), 7.0, dtype=s.dt, device="cuda")
    torch.cuda.synchronize()
    pw.pw_attn_forward(s.attn, 0, 0, s.q, o)
    with pytest.raises(pw.PwError) as e:
        pw.pw_attn_check(s.attn)
    assert e.value.status == pw.PW_ERR_STATE and bool((o == 7.0).all())
    graph.replay()
    torch.cuda.synchronize()
    s.compare()
    s.close()


def test_a_whole_step_with_groups_in_a_graph_follows_the_lengths():
    import torch
    s = Step([100, 90, 85, 120], [1, 1, 1, 1], Hq=4, Hkv=2, D=128, dtype="fp16", group_start=[0, 4], prefix=80, spare_ids=4)
    s.map_and_append()
    s.compare()
    o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        s.pw.pw_kv_map(s.attn, s.step, s.new_ids, stream=stream)
        s.pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v, stream=stream)
        s.pw.pw_attn_plan(s.attn, 0, s.step, stream=stream)
        s.pw.pw_attn_forward(s.attn, 0, 0, s.q, o, stream=stream)
    for ctx, new in (([100, 90, 85, 120], [1, 1, 1, 1]), ([81, 90, 80, 99], [1, 0, 2, 1]), ([99, 85, 84, 111], [0, 1, 1, 1])):
        s.ctx, s.new = ctx, new
        s.step.refs[0].copy_(torch.tensor(ctx, dtype=torch.int32))
        s.step.refs[1].copy_(torch.tensor(new, dtype=torch.int32))
        s.table.copy_(torch.as_tensor(s.table0))  # (without the blocks that an earlier replay opened)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s.pw.pw_attn_check(s.attn)
        want, _, absum, _, where = s.expect()
        n, got = len(where), o.float().cpu().numpy()
        assert (np.abs(got[:n] - want) <= UNIT["fp16"] * (np.abs(want) + absum) + 1e-4 * absum + 1e-6).all()
        assert not got[n:].any()
    s.close()
