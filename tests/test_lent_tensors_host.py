"""Tensors of calls on a stream that is not torch's current one are lent to it, with stand-ins for tensors and library."""
from types import SimpleNamespace

import pytest
import torch

from test_attn_binding_host import On

pw = pytest.importorskip("any_precision_bit_gb300")


class Lent(On):
    """A CPU tensor that says it is on a GPU and notes the streams it is lent to."""

    def __init__(self, *a):
        super().__init__(*a)
        self.lent = []

    def record_stream(self, stream):
        self.lent.append(stream)


class Agrees:
    def __getattr__(self, name):
        return lambda *a: 0


def ints(n, dtype=torch.int32):
    return Lent(torch.zeros(n, dtype=dtype), 1)


def floats(*n):
    return Lent(torch.zeros(*n), 1)


def rows(h):
    return Lent(torch.zeros(4, h, 8, dtype=torch.bfloat16), 1)


def calls():
    """(call(stream), its tensors) of every asynchronous call; the step's tensors are among them."""
    s = dict(ctx_len=ints(2), new_len=ints(2), table=ints((2, 3)), q_start=ints(3), kv_len=ints(2), slot=ints(4, torch.int64),
             pos=ints(4), rows=ints(2), groups=ints(2), shared_len=ints(1))
    step, mine = pw.pw_make_step(**s, max_new=2), list(s.values())
    ids, doc, two = ints(1), ints(4), ints(2)
    yield lambda st: pw.pw_kv_map(7, step, ids, stream=st), [ids, *mine]
    yield lambda st: pw.pw_attn_plan(7, 0, step, doc_start=doc, bidir_len=two, stream=st), [doc, two, *mine]
    q, o, k, v, lse, slopes = rows(4), rows(4), rows(2), rows(2), floats(4, 4), floats(4)
    yield lambda st: pw.pw_attn_append(7, 0, step, k, v, stream=st), [k, v, *mine]
    yield lambda st: pw.pw_attn_forward(7, 0, 0, q, o, lse=lse, slopes=slopes, stream=st), [q, o, lse, slopes, *mine]
    pos, length, parent, n, ctx = ints(8), ints(2), ints((2, 3)), ints(2), ints(2)
    yield lambda st: pw.pw_attn_rope_append(7, 0, step, q, o, k, v, pos=pos, stream=st), [q, o, k, v, pos, *mine]
    yield lambda st: pw.pw_attn_plan_tree(7, 0, step, length, parent, pos=doc, stream=st), [length, parent, doc, *mine]
    yield lambda st: pw.pw_attn_forward(7, 0, 0, q, o, stream=st), [q, o, length, parent, doc, *mine]
    yield lambda st: pw.pw_kv_keep(7, step, length, parent, n, ctx_out=ctx, stream=st), [length, parent, n, ctx, *mine]
    table = ints((2, 3))
    yield lambda st: pw.pw_kv_copy(7, two, n, table=table, stream=st), [two, n, table]


@pytest.mark.parametrize("current", [0, 5])
def test_tensors_are_lent_to_a_stream_that_is_not_current(monkeypatch, current):
    desc = pw.pw_attn_desc(L=1, n_heads=4, n_kv_heads=2, head_dim=8, dtype=pw.PW_BF16, n_blocks=3, block_tokens=16,
                           max_requests=2, max_tokens=4, max_shared_tokens=4, n_plans=1, device=1, max_tree_tokens=4)
    pw._load_types()
    monkeypatch.setattr(pw, "lib", Agrees)
    monkeypatch.setattr(pw, "_raw_stream", lambda device: current if device == 1 else pytest.fail("another device"))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: (raw, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: (0, device))
    monkeypatch.setitem(pw._attn_shapes, 7, (4, 2, 8, torch.bfloat16, 1, desc, {}, {}))
    monkeypatch.setitem(pw._rope_axes, (7, 0), 2)
    other = SimpleNamespace(cuda_stream=9)
    default = (0, 1) if current else None
    for call, tensors in calls():
        for stream, lent in ((other, other), (9, (9, 1)), (pw.C.c_void_p(9), (9, 1)), (None, default), (0, default),
                             (SimpleNamespace(cuda_stream=current), None), (current, None)):
            for t in tensors:
                t.lent.clear()
            call(stream)
            for t in tensors:
                assert t.lent == ([] if lent is None else [lent])
