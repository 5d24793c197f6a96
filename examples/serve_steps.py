"""A small serving loop over the library's calls: requests that share a system prompt come in
with prompts of their own, and then decode, through layers of paged attention and
mixed-precision experts.

Per step the KV-block allocator (pw_kv_*) grants the blocks that the new tokens open, pw_kv_map
turns lengths and grants into block tables and slots on the device, and pw_attn_plan lays out
the attention; per layer the projections (torch), pw_attn_append, pw_attn_forward and
pw_moe_forward run on one stream.  Weights are random and the "sampling" a fixed map: the loop
shows how the calls fit together.

    python examples/serve_steps.py
"""
from __future__ import annotations

import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import any_precision_bit_gb300 as pw  # noqa: E402
import synthetic as syn  # noqa: E402

LAYERS, N_HEADS, N_KV_HEADS, HEAD_DIM, BLOCK = 2, 8, 2, 32, 16
WINDOW = 40  # layer 1 attends to the last WINDOW positions, layer 0 to all


class Server:
    def __init__(self, system_tokens, max_requests, max_tokens, n_blocks, seed=0):
        self.shape = sh = syn.SHAPES["tiny"]
        self.dev, self.H = torch.device("cuda:0"), sh.H
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16).to(self.dev)  # noqa: E731
        width = N_HEADS * HEAD_DIM
        self.wqkv = [w(width + 2 * N_KV_HEADS * HEAD_DIM, sh.H) for _ in range(LAYERS)]
        self.wo = [w(sh.H, width) for _ in range(LAYERS)]
        # experts
        self.moe = pw.pw_create(pw.pw_desc(L=LAYERS, E=sh.E, H=sh.H, I=sh.I, K=sh.K, Is=0, bmax=sh.bmax,
                                           bits_mask=sh.bits_mask(), renorm=0, device=0, max_tokens=max_tokens, flags=0))
        for layer in range(LAYERS):
            Wr, bias, _ = syn.gen_router_np(sh, seed, layer)
            pw.pw_set_router(self.moe, layer, Wr, bias)
            q = syn.gen_q_assignment(sh, seed, layer)
            for e in range(sh.E):
                for u in (0, 1):
                    idx, luts = syn.gen_block_np(sh, seed, layer, e, u)
                    pw.pw_pack(self.moe, layer, e, u, idx, np.concatenate([luts[b].ravel() for b in sh.bits]), int(q[e, u]))
        # cache, its allocator (one budget with the weight pages) and the attention handle
        shape = (LAYERS, 2, n_blocks, BLOCK, N_KV_HEADS, HEAD_DIM)
        self.cache = torch.empty(shape, dtype=torch.bfloat16, device=self.dev)
        block_bytes = LAYERS * 2 * BLOCK * N_KV_HEADS * HEAD_DIM * 2
        self.kv = pw.pw_kv_create(pw.pw_memory(self.moe).held_bytes + n_blocks * block_bytes, block_bytes)
        pw.pw_kv_attach(self.kv, self.moe)
        self.attn = pw.pw_attn_create(pw.pw_attn_desc(
            L=LAYERS, n_heads=N_HEADS, n_kv_heads=N_KV_HEADS, head_dim=HEAD_DIM, dtype=pw.PW_BF16, n_blocks=n_blocks,
            block_tokens=BLOCK, max_requests=max_requests, max_tokens=max_tokens, max_shared_tokens=max_tokens, n_plans=2,
            device=0))
        for layer in range(LAYERS):
            pw.pw_attn_bind(self.attn, layer, self.cache[layer, 0], self.cache[layer, 1])
        self.table = torch.full((max_requests, n_blocks), -1, dtype=torch.int32, device=self.dev)
        self.length = {}  # tokens in the cache, by request; a request's table row is its index here
        self.stream = torch.cuda.Stream()
        # the system prompt, request -1 of the allocator: its blocks head the tables of all requests
        self.system = system_tokens // BLOCK * BLOCK
        if self.system:
            self.stream.wait_stream(torch.cuda.current_stream())  # the table is filled
            with torch.cuda.stream(self.stream):
                x = torch.randn(self.system, sh.H, generator=g).to(torch.bfloat16).to(self.dev)
                self._step([0], [0], [self.system], x, keys=[-1], share=False)
            self.table[1:, :self.system // BLOCK] = self.table[0, :self.system // BLOCK]
            torch.cuda.synchronize()

    def admit(self, request):
        self.length[request] = self.system

    def _i32(self, a):
        return torch.tensor(a, dtype=torch.int32).to(self.dev, non_blocking=True)

    def _step(self, rows, ctx, new, x, keys, share=True):
        """One engine step of requests with `ctx` cached and `new` new tokens, x their hidden states."""
        grants = []
        for key, c, n in zip(keys, ctx, new):
            grants.append(pw.pw_kv_grow(self.kv, key, -(-(c + n) // BLOCK) - -(-c // BLOCK)))
        ids = self._i32(np.concatenate(grants)) if sum(map(len, grants)) else None
        N, R, dev = sum(new), len(new), self.dev
        empty = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device=dev)  # noqa: E731
        shared = share and self.system > 0
        step = pw.pw_make_step(self._i32(ctx), self._i32(new), self.table, empty(R + 1), empty(R), empty(N, torch.int64),
                               empty(N), max_new=max(new), rows=self._i32(rows),
                               groups=self._i32([0, R]) if shared else None,
                               shared_len=self._i32([self.system]) if shared else None)
        s = self.stream
        pw.pw_kv_map(self.attn, step, ids, stream=s)
        pw.pw_attn_plan(self.attn, 0, step, stream=s)
        pw.pw_attn_plan(self.attn, 1, step, window=WINDOW, stream=s)
        nq, nk = N_HEADS * HEAD_DIM, N_KV_HEADS * HEAD_DIM
        o = torch.empty(N, N_HEADS, HEAD_DIM, dtype=torch.bfloat16, device=dev)
        for layer in range(LAYERS):
            norm = x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)
            qkv = norm.to(x.dtype) @ self.wqkv[layer].T
            q = qkv[:, :nq].view(N, N_HEADS, HEAD_DIM)
            k = qkv[:, nq:nq + nk].view(N, N_KV_HEADS, HEAD_DIM)
            v = qkv[:, nq + nk:].view(N, N_KV_HEADS, HEAD_DIM)
            pw.pw_attn_append(self.attn, layer, step, k, v, stream=s)
            pw.pw_attn_forward(self.attn, layer, layer % 2, q, o, softcap=30.0, stream=s)
            x = (x + o.view(N, nq) @ self.wo[layer].T).contiguous()
            pw.pw_moe_forward(self.moe, layer, x, N, x, flags=pw.PW_ACCUMULATE | pw.PW_PRENORM, stream=s)
        pw.pw_attn_check(self.attn, s)  # waits for the stream; the step's tensors may go
        pw.pw_check(self.moe)
        return x

    def step(self, hidden):
        """hidden: {request: bf16 [new][H]}; the outputs, likewise, complete on return."""
        self.stream.wait_stream(torch.cuda.current_stream())  # where the hidden states were made
        names = list(hidden)
        new = [hidden[r].shape[0] for r in names]
        with torch.cuda.stream(self.stream):
            x = torch.cat([hidden[r] for r in names])
            y = self._step([list(self.length).index(r) for r in names], [self.length[r] for r in names], new, x, keys=names)
        for r, n in zip(names, new):
            self.length[r] += n
        return dict(zip(names, y.split(new)))

    def close(self):
        torch.cuda.synchronize()
        for r in [-1, *self.length]:
            pw.pw_kv_release(self.kv, r)
        pw.pw_kv_destroy(self.kv)
        pw.pw_attn_destroy(self.attn)
        pw.pw_destroy(self.moe)


def main(system_tokens=80, prompts=(13, 1, 50), decode_steps=4, seed=0):
    """Outputs of every step, request by request: {request: [tensor per step]}."""
    server = Server(system_tokens, max_requests=8, max_tokens=256, n_blocks=64, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    out = {}
    hidden = {}
    for r, n in enumerate(prompts):
        server.admit(r)
        out[r] = []
        hidden[r] = torch.randn(n, server.H, generator=g).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    for _ in range(1 + decode_steps):
        for r, y in server.step(hidden).items():
            out[r].append(y.float().cpu())
            hidden[r] = torch.roll(y[-1:], 1, dims=1)  # the next token's hidden state
    stats = pw.pw_kv_get_stats(server.kv)
    server.close()
    return out, stats


if __name__ == "__main__":
    outputs, stats = main()
    for r, steps in outputs.items():
        print(f"request {r}: prompt {steps[0].shape[0]} tokens, then {len(steps) - 1}; last state rms "
              f"{steps[-1].pow(2).mean().sqrt():.4f}")
    print(f"KV blocks used {stats['used_blocks']} of {stats['capacity_blocks']}")
