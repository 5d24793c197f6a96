"""The new attention calls' checks of where a tensor lies and of their arguments, without a GPU."""
import numpy as np
import pytest
import torch

from test_attn_binding_host import NoLibrary, On, ints, step

pw = pytest.importorskip("any_precision_bit_gb300")


@pytest.fixture(scope="module", autouse=True)
def built():
    from any_precision_bit_gb300 import _build
    _build.build()


@pytest.mark.parametrize("n", [-1, 9])
def test_create_refuses(n):
    with pytest.raises(pw.PwError) as e:
        pw.pw_attn_create(pw.pw_attn_desc(L=1, n_heads=4, n_kv_heads=2, head_dim=64, dtype=0, n_blocks=10, block_tokens=16,
                                          max_requests=2, max_tokens=8, max_shared_tokens=0, n_plans=1, device=0,
                                          max_tree_tokens=n))
    assert e.value.status == pw.PW_ERR_INVALID and "max_tree_tokens" in str(e.value)


def test_null_handles_are_refused():
    lib = pw.lib()
    assert lib.pw_attn_set_rope(None, 0, None) == pw.PW_ERR_INVALID
    assert lib.pw_attn_rope_append(*[None, 0, None, None, 0, 0, None, 0, 0, None, 0, 0, None, 0, 0, None, None]) == pw.PW_ERR_INVALID
    assert lib.pw_attn_plan_tree(None, 0, None, 0, None, None) == pw.PW_ERR_INVALID
    assert lib.pw_kv_keep(None, None, None, None, 0, None, None, None) == pw.PW_ERR_INVALID
    assert lib.pw_kv_copy(None, None, None, 0, None, 0, 0, None) == pw.PW_ERR_INVALID


def test_calls_refuse_tensors_of_another_device_than_the_handle(monkeypatch):
    desc = pw.pw_attn_desc(L=1, n_heads=4, n_kv_heads=2, head_dim=8, dtype=pw.PW_BF16, n_blocks=3, block_tokens=16,
                           max_requests=2, max_tokens=4, max_shared_tokens=0, n_plans=1, device=1, max_tree_tokens=4)
    monkeypatch.setattr(pw, "lib", NoLibrary)
    here = step()
    monkeypatch.setitem(pw._attn_shapes, 7, (4, 2, 8, torch.bfloat16, 1, desc, {}, {}))
    monkeypatch.setitem(pw._rope_axes, (7, 0), 2)
    there = step(**{k: ints(n, 0) for k, n in dict(ctx_len=2, new_len=2, table=(2, 3), q_start=3, kv_len=2, pos=4, rows=2,
                                                   groups=2, shared_len=1).items()},
                 slot=On(torch.zeros(4, dtype=torch.int64), 0))

    def rows(h, device=1, dtype=torch.bfloat16):
        return On(torch.zeros(4, h, 8, dtype=dtype), device)

    def rope(**kw):
        a = {**dict(step=here, q=rows(4), q_out=rows(4), k=rows(2), v=rows(2), pos=None), **kw}
        return lambda: pw.pw_attn_rope_append(7, 0, a["step"], a["q"], a["q_out"], a["k"], a["v"], pos=a["pos"])

    def tree(**kw):
        a = {**dict(step=here, tree_len=ints(2), parent=ints((2, 3)), pos=ints(4)), **kw}
        return lambda: pw.pw_attn_plan_tree(7, 0, a["step"], a["tree_len"], a["parent"], pos=a["pos"])

    def keep(**kw):
        a = {**dict(step=here, tree_len=ints(2), keep=ints((2, 3)), n_keep=ints(2), ctx_out=ints(2)), **kw}
        return lambda: pw.pw_kv_keep(7, a["step"], a["tree_len"], a["keep"], a["n_keep"], ctx_out=a["ctx_out"])

    def copy(**kw):
        a = {**dict(src=ints(2), dst=ints(2), table=ints((2, 3))), **kw}
        return lambda: pw.pw_kv_copy(7, a["src"], a["dst"], table=a["table"])

    calls = [rope(step=there), rope(q=rows(4, 0)), rope(q_out=rows(4, 0)), rope(k=rows(2, 0)), rope(v=rows(2, 0)),
             rope(v=rows(2, dtype=torch.float16)), rope(q_out=rows(2)), rope(pos=ints(8, 0)), rope(pos=ints(7)), rope(pos=ints((4, 2))),
             tree(step=there), tree(tree_len=ints(2, 0)), tree(parent=ints((2, 3), 0)), tree(pos=ints(4, 0)), tree(pos=ints(3)),
             tree(parent=ints((1, 3))), tree(parent=ints(6)), keep(keep=ints(6)),
             keep(step=there), keep(tree_len=ints(1)), keep(keep=ints((2, 3), 0)), keep(n_keep=ints(2, 0)), keep(ctx_out=ints(1)),
             copy(src=ints(2, 0)), copy(dst=ints(1)), copy(dst=ints(2, 0)), copy(table=ints((2, 3), 0)),
             lambda: pw.pw_attn_set_rope(7, 0, [1.0] * 4, axis=[0] * 3), lambda: pw.pw_attn_set_rope(7, 0, [1.0] * 4, q_gain=np.ones(7)),
             lambda: pw.pw_attn_set_rope(7, 0, [1.0] * 4, k_gain=On(torch.ones(8), 0))]
    for call in calls:
        with pytest.raises(ValueError):
            call()
