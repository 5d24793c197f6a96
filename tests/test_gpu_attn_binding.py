"""The binding's checks of the tensors' types, and the references that it keeps."""
import gc

import numpy as np
import pytest

from attn_helpers import Step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_tensors_of_another_type_of_the_same_size_are_refused(dtype):
    import torch
    s = Step([20, 7], [2, 3], D=64, dtype=dtype)
    pw = s.pw
    s.map_and_append()
    pw.pw_attn_plan(s.attn, 0, s.step)
    o = torch.empty(s.N, s.Hq, s.D, dtype=s.dt, device="cuda")
    lse, slopes = torch.empty(s.N, s.Hq, device="cuda"), torch.ones(s.Hq, device="cuda")
    ints, reals = torch.zeros(s.N, dtype=torch.int32, device="cuda"), torch.zeros(s.N, device="cuda")
    step = dict(ctx_len=ints[:2], new_len=ints[:2], table=s.table, q_start=s.q_start, kv_len=s.kv_len, slot=s.slot, pos=s.pos)

    def make(**change):
        return pw.pw_make_step(**{**step, **change}, max_new=3)

    wrong = []
    for other in (torch.float16 if dtype == "bf16" else torch.bfloat16, torch.int16):
        wrong += [
            lambda t=other: pw.pw_attn_bind(s.attn, 0, s.kv[0].view(t), s.kv[1].view(t)),
            lambda t=other: pw.pw_attn_bind(s.attn, 0, s.kv[0], s.kv[1].view(t)),
            lambda t=other: pw.pw_attn_append(s.attn, 0, s.step, s.k.view(t), s.v),
            lambda t=other: pw.pw_attn_append(s.attn, 0, s.step, s.k, s.v.view(t)),
            lambda t=other: pw.pw_attn_forward(s.attn, 0, 0, s.q.view(t), o),
            lambda t=other: pw.pw_attn_forward(s.attn, 0, 0, s.q, o.view(t)),
        ]
    wrong += [
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o, lse=lse.view(torch.int32)),
        lambda: pw.pw_attn_forward(s.attn, 0, 0, s.q, o, slopes=slopes.view(torch.int32)),
        lambda: pw.pw_attn_plan(s.attn, 0, s.step, doc_start=reals),
        lambda: pw.pw_attn_plan(s.attn, 0, s.step, bidir_len=reals[:2]),
        lambda: pw.pw_kv_map(s.attn, s.step, s.new_ids.view(torch.float32)),
        lambda: make(ctx_len=reals[:2]), lambda: make(new_len=reals[:2]), lambda: make(table=s.table.view(torch.float32)),
        lambda: make(q_start=s.q_start.view(torch.float32)), lambda: make(kv_len=reals[:2]),
        lambda: make(slot=s.slot.view(torch.float64)), lambda: make(pos=s.pos.view(torch.float32)),
        lambda: make(rows=reals[:2]), lambda: make(groups=reals[:2], shared_len=ints[:1]),
        lambda: make(groups=ints[:2], shared_len=reals[:1]),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} went through")
    make()
    s.compare()
    s.close()


def test_a_plan_keeps_its_step_and_a_binding_its_caches():
    """The caller's references may go: the table and the caches stay until another step is planned, others are
    bound, or the handle is destroyed."""
    import torch
    import weakref
    s = Step([100, 40], [1, 2], D=64, n_plans=2)
    pw = s.pw
    s.map_and_append()
    want = s.forward()
    kept = [weakref.ref(s.table), weakref.ref(s.kv[0]), weakref.ref(s.kv[1])]
    q, attn, ctx, shapes = s.q, s.attn, (s.N, s.Hq, s.D), [c.shape for c in s.kv]
    pw.pw_attn_plan(attn, 1, s.step)
    new = dict(ctx_len=s.step.refs[0], new_len=s.step.refs[1], table=s.table.clone(), q_start=s.q_start, kv_len=s.kv_len,
               slot=s.slot, pos=s.pos, max_new=2)
    s.table = s.kv = s.step = None
    gc.collect()
    assert all(r() is not None for r in kept)
    junk = [torch.full(sh, float("nan"), dtype=s.dt, device="cuda") for sh in shapes for _ in range(4)]
    o = torch.empty(*ctx, dtype=s.dt, device="cuda")
    pw.pw_attn_forward(attn, 0, 0, q, o)
    pw.pw_attn_check(attn)
    assert np.array_equal(o.float().cpu().numpy(), want[0])
    step = pw.pw_make_step(**new)
    pw.pw_attn_plan(attn, 0, step)
    gc.collect()
    assert kept[0]() is not None  # plan 1 still has it
    pw.pw_attn_plan(attn, 1, step)
    gc.collect()
    assert kept[0]() is None
    pw.pw_attn_check(attn)
    pw.pw_attn_bind(attn, 0, *[j for j in junk[:2]])
    gc.collect()
    assert kept[1]() is None and kept[2]() is None
    table = weakref.ref(new.pop("table"))
    junk = weakref.ref(junk.pop(0))
    pw.pw_attn_destroy(attn)
    step = None
    gc.collect()
    assert table() is None and junk() is None
