"""examples/serve_steps.py: allocator, maps, cache, attention and experts as a server calls them."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def serve():
    from any_precision_bit_gb300 import _build
    _build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_steps
    return serve_steps


def test_runs_and_repeats(serve):
    import torch
    a, stats = serve.main()
    b, _ = serve.main()
    assert stats["used_blocks"] == 5 + sum(-(-(80 + n + 4) // 16) - 5 for n in (13, 1, 50))
    for r in a:
        assert len(a[r]) == 5
        for x, y in zip(a[r], b[r]):
            assert torch.isfinite(x).all() and torch.equal(x, y)


def test_token_by_token_is_the_prompt_at_once(serve):
    """The same hidden states as a prompt and single tokens, or all in one step: outputs of each token
    within the rounding of two bf16 layers (3 %), but for the few whose experts are so nearly tied that
    this rounding chooses others."""
    import torch
    g = torch.Generator().manual_seed(7)
    x = torch.randn(37, 128, generator=g).to(torch.bfloat16).cuda()
    out = []
    for cuts in ([37], [20, 1, 1, 9, 1, 5]):
        s = serve.Server(48, max_requests=4, max_tokens=64, n_blocks=32)
        s.admit(0)
        torch.cuda.synchronize()
        out.append(torch.cat([s.step({0: part.contiguous()})[0].float() for part in x.split(cuts)]))
        s.close()
    err = (out[0] - out[1]).norm(dim=1) / out[0].norm(dim=1)
    assert (err < 0.03).float().mean() >= 0.8 and err.max() < 1.0, err


def test_inputs_that_another_stream_is_still_writing(serve):
    """Hidden states made on the caller's current stream just before the call are waited for."""
    import torch
    g = torch.Generator().manual_seed(7)
    x = torch.randn(5, 128, generator=g).to(torch.bfloat16).cuda()
    out = []
    for late in (False, True):
        s = serve.Server(48, max_requests=4, max_tokens=64, n_blocks=32)
        s.admit(0)
        h = torch.zeros_like(x)
        torch.cuda.synchronize()
        if late:
            torch.cuda._sleep(100_000_000)  # about 50 ms
        h.copy_(x)
        out.append(s.step({0: h})[0].float())
        s.close()
    assert torch.equal(out[0], out[1])


@pytest.mark.parametrize("cuts", [[37], [20, 1, 1, 1, 9, 1, 1, 1, 2], [5] + [1] * 32])
def test_attention_of_every_token_is_the_formula(serve, monkeypatch, cuts):
    """Layer 0 of the example, whose attention comes before any expert: its outputs for every token of a prompt that
    comes in parts, against float64 over all keys of the system prompt and the tokens before.  One rounding of each
    probability and one of the result (2^-8 each), and 1e-4 for the fp32 steps."""
    import numpy as np
    import torch
    seen = {"k": [], "v": [], "q": [], "o": []}
    append, forward = serve.pw.pw_attn_append, serve.pw.pw_attn_forward

    def keep(name, t):
        seen[name].append(t.float().cpu().numpy().astype(np.float64))

    def record_append(attn, layer, step, k, v, stream=None):
        append(attn, layer, step, k, v, stream=stream)
        if layer == 0:
            keep("k", k), keep("v", v)

    def record_forward(attn, layer, plan, q, o, stream=None, **kw):
        forward(attn, layer, plan, q, o, stream=stream, **kw)
        if layer == 0:
            assert kw == dict(softcap=30.0)
            keep("q", q), keep("o", o)

    monkeypatch.setattr(serve.pw, "pw_attn_append", record_append)
    monkeypatch.setattr(serve.pw, "pw_attn_forward", record_forward)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(37, 128, generator=g).to(torch.bfloat16).cuda()
    s = serve.Server(48, max_requests=4, max_tokens=64, n_blocks=32)
    s.admit(0)
    for part in x.split(cuts):
        s.step({0: part.contiguous()})
    s.close()
    k, v, q, o = (np.concatenate(seen[n]) for n in "kvqo")
    assert len(k) == len(o) == 48 + 37
    for t in range(48 + 37):
        for h in range(serve.N_HEADS):
            kv = h * serve.N_KV_HEADS // serve.N_HEADS
            y = 30.0 * np.tanh(k[:t + 1, kv] @ q[t, h] / serve.HEAD_DIM ** 0.5 / 30.0)
            p = np.exp(y - y.max())
            p /= p.sum()
            want, size = p @ v[:t + 1, kv], p @ np.abs(v[:t + 1, kv])
            assert (np.abs(o[t, h] - want) <= 2.0 ** -8 * (np.abs(want) + size) + 1e-4 * size).all(), (t, h)
