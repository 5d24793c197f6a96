"""The attention binding's checks of where a tensor lies, with stand-ins for tensors of several GPUs."""
import pytest
import torch

pw = pytest.importorskip("any_precision_bit_gb300")


class On:
    """A CPU tensor that says it is on a GPU."""

    def __init__(self, t, device):
        self.t, self.index, self.device = t, device, f"cuda:{device}"

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class NoLibrary:
    def __getattr__(self, name):
        return lambda *a: pytest.fail(f"{name} was called")


def ints(n, device=1, **kw):
    return On(torch.zeros(n, dtype=torch.int32, **kw), device)


def step(**change):
    kw = dict(ctx_len=ints(2), new_len=ints(2), table=ints((2, 3)), q_start=ints(3), kv_len=ints(2),
              slot=On(torch.zeros(4, dtype=torch.int64), 1), pos=ints(4), rows=ints(2), groups=ints(2), shared_len=ints(1))
    return pw.pw_make_step(**{**kw, **change}, max_new=2)


def test_a_step_is_on_one_device():
    assert step().device == 1
    other = dict(new_len=ints(2, 0), table=ints((2, 3), 0), q_start=ints(3, 0), kv_len=ints(2, 0),
                 slot=On(torch.zeros(4, dtype=torch.int64), 0), pos=ints(4, 0), rows=ints(2, 0), groups=ints(2, 0),
                 shared_len=ints(1, 0), ctx_len=ints(2, 0))
    for name, t in other.items():
        with pytest.raises(ValueError):
            step(**{name: t})
    with pytest.raises(ValueError):
        step(ctx_len=torch.zeros(2, dtype=torch.int32))


def test_calls_refuse_tensors_of_another_device_than_the_handle(monkeypatch):
    desc = pw.pw_attn_desc(L=1, n_heads=4, n_kv_heads=2, head_dim=8, dtype=pw.PW_BF16, n_blocks=3, block_tokens=16,
                           max_requests=2, max_tokens=4, max_shared_tokens=0, n_plans=1, device=1)
    monkeypatch.setattr(pw, "lib", NoLibrary)
    step()  # (loads the types)
    monkeypatch.setitem(pw._attn_shapes, 7, (4, 2, 8, torch.bfloat16, 1, desc, {}, {}))

    def rows(h, device=1, dtype=torch.bfloat16):
        return On(torch.zeros(4, h, 8, dtype=dtype), device)

    here, there = step(), step(**{k: ints(n, 0) for k, n in dict(ctx_len=2, new_len=2, table=(2, 3), q_start=3, kv_len=2, pos=4,
                                                                rows=2, groups=2, shared_len=1).items()},
                               slot=On(torch.zeros(4, dtype=torch.int64), 0))
    cache = torch.zeros(3, 16, 2, 8, dtype=torch.bfloat16)
    calls = [
        lambda: pw.pw_kv_map(7, there, None), lambda: pw.pw_kv_map(7, here, ints(1, 0)),
        lambda: pw.pw_attn_plan(7, 0, there), lambda: pw.pw_attn_plan(7, 0, here, doc_start=ints(4, 0)),
        lambda: pw.pw_attn_plan(7, 0, here, bidir_len=ints(2, 0)),
        lambda: pw.pw_attn_append(7, 0, there, rows(2), rows(2)), lambda: pw.pw_attn_append(7, 0, here, rows(2, 0), rows(2)),
        lambda: pw.pw_attn_append(7, 0, here, rows(2), rows(2, 0)),
        lambda: pw.pw_attn_append(7, 0, here, rows(2), rows(2, dtype=torch.float16)),
        lambda: pw.pw_attn_forward(7, 0, 0, rows(4, 0), rows(4)), lambda: pw.pw_attn_forward(7, 0, 0, rows(4), rows(4, 0)),
        lambda: pw.pw_attn_forward(7, 0, 0, rows(4), rows(4), lse=On(torch.zeros(16), 0)),
        lambda: pw.pw_attn_forward(7, 0, 0, rows(4), rows(4), slopes=On(torch.zeros(4), 0)),
        lambda: pw.pw_attn_bind(7, 0, On(cache, 0), On(cache, 1)), lambda: pw.pw_attn_bind(7, 0, On(cache, 1), On(cache, 0)),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
