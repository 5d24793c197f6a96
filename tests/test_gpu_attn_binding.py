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
