"""Drafted trees over the paged cache: each step verifies a tree of guesses for every request and keeps the path that the
model agrees with; a request is forked, another one ends, and the cache is compacted in between.

Per step pw_kv_grow grants blocks for all nodes, pw_kv_map and pw_attn_plan_tree turn lengths and parents into slots, masks
and positions on the device; per layer pw_attn_rope_append norms and turns queries and keys and writes the cache, and
pw_attn_forward attends.  Behind the step pw_kv_keep moves the accepted nodes' keys and values together and pw_kv_trim
returns the blocks of the others.  Weights are random, the draft "model" is the embedding alone, and sampling is greedy: the
loop shows how the calls fit together.

    python examples/draft_steps.py
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

LAYERS, HIDDEN, N_HEADS, N_KV_HEADS, HEAD_DIM, BLOCK, VOCAB = 2, 128, 8, 2, 32, 16, 64
WIDTHS = (3, 2, 1, 1)  # children of a node, by depth


class Server:
    def __init__(self, max_requests, max_tokens, n_blocks, seed=0):
        self.dev = torch.device("cuda:0")
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(*s, generator=g) / s[-1] ** 0.5).to(torch.bfloat16).to(self.dev)  # noqa: E731
        width = N_HEADS * HEAD_DIM
        self.emb = torch.randn(VOCAB, HIDDEN, generator=g).to(torch.bfloat16).to(self.dev)
        self.head = w(VOCAB, HIDDEN)
        self.wqkv = [w(width + 2 * N_KV_HEADS * HEAD_DIM, HIDDEN) for _ in range(LAYERS)]
        self.wo = [0.5 * w(HIDDEN, width) for _ in range(LAYERS)]
        self.guess = (self.emb.float() @ self.head.float().T).argsort(-1, descending=True).cpu()  # the drafts' next tokens
        self.cache = torch.empty(LAYERS, 2, n_blocks, BLOCK, N_KV_HEADS, HEAD_DIM, dtype=torch.bfloat16, device=self.dev)
        self.kv = pw.pw_kv_create(n_blocks, 1)
        self.attn = pw.pw_attn_create(pw.pw_attn_desc(
            L=LAYERS, n_heads=N_HEADS, n_kv_heads=N_KV_HEADS, head_dim=HEAD_DIM, dtype=pw.PW_BF16, n_blocks=n_blocks,
            block_tokens=BLOCK, max_requests=max_requests, max_tokens=max_tokens, n_plans=1, device=0, max_tree_tokens=max_tokens))
        inv_freq = 10000.0 ** (-np.arange(0, HEAD_DIM, 2) / HEAD_DIM)
        for layer in range(LAYERS):
            pw.pw_attn_bind(self.attn, layer, self.cache[layer, 0], self.cache[layer, 1])
            gain = 1 + 0.1 * torch.randn(2, HEAD_DIM, generator=g)
            pw.pw_attn_set_rope(self.attn, layer, inv_freq, q_gain=gain[0], k_gain=gain[1])
        self.table = torch.full((max_requests, n_blocks), -1, dtype=torch.int32, device=self.dev)
        self.free_rows = list(range(max_requests))
        self.row, self.ctx, self.tokens = {}, {}, {}  # table row, tokens in the cache, and all tokens, by request
        self.seen = {}  # last hidden state of every token that is in the cache, for whoever wants to check them

    def _i32(self, a):
        return torch.as_tensor(np.asarray(a), dtype=torch.int32).to(self.dev)

    def _forward(self, names, tokens, parents):
        """One step with the new tokens of every request; parents of its nodes, or None for a prompt.  Returns the step,
        the trees' lengths and the last hidden states."""
        new = [len(t) for t in tokens]
        ctx = [self.ctx[r] for r in names]
        grants = [pw.pw_kv_grow(self.kv, r, -(-(c + n) // BLOCK) - -(-c // BLOCK)) for r, c, n in zip(names, ctx, new)]
        N, R = sum(new), len(new)
        empty = lambda n, dt=torch.int32: torch.empty(n, dtype=dt, device=self.dev)  # noqa: E731
        step = pw.pw_make_step(self._i32(ctx), self._i32(new), self.table, empty(R + 1), empty(R), empty(N, torch.int64), empty(N),
                               max_new=max(new), rows=self._i32([self.row[r] for r in names]))
        tree_len = self._i32([0 if p is None else len(p) for p in parents])
        flat = np.full((R, max([1] + [len(p) for p in parents if p is not None])), -1)
        for r, p in enumerate(parents):
            flat[r, :len(p or [])] = p or []
        s, pos, parent = torch.cuda.current_stream(), empty(N), self._i32(flat)
        pw.pw_kv_map(self.attn, step, self._i32(np.concatenate(grants)), stream=s)
        pw.pw_attn_plan_tree(self.attn, 0, step, tree_len, parent, pos=pos, stream=s)
        x = self.emb[torch.as_tensor(sum(tokens, []), device=self.dev)]
        nq, nk = N_HEADS * HEAD_DIM, N_KV_HEADS * HEAD_DIM
        o = torch.empty(N, N_HEADS, HEAD_DIM, dtype=torch.bfloat16, device=self.dev)
        for layer in range(LAYERS):
            norm = x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)
            qkv = norm.to(x.dtype) @ self.wqkv[layer].T
            q = qkv[:, :nq].view(N, N_HEADS, HEAD_DIM)
            k = qkv[:, nq:nq + nk].view(N, N_KV_HEADS, HEAD_DIM)
            v = qkv[:, nq + nk:].view(N, N_KV_HEADS, HEAD_DIM)
            pw.pw_attn_rope_append(self.attn, layer, step, q, q, k, v, pos=pos, stream=s)
            pw.pw_attn_forward(self.attn, layer, 0, q, o, stream=s)
            x = x + o.view(N, nq) @ self.wo[layer].T
        pw.pw_attn_check(self.attn, s)
        return step, tree_len, x

    def _next(self, x):
        return (x.float() @ self.head.float().T).argmax(-1).tolist()

    def admit(self, request, prompt):
        """Run a prompt; its next token is known then, and not yet in the cache."""
        self.row[request], self.ctx[request] = self.free_rows.pop(0), 0
        _, _, x = self._forward([request], [prompt], [None])
        self.ctx[request] = len(prompt)
        self.tokens[request] = [*prompt, self._next(x[-1:])[0]]
        self.seen[request] = list(x.float().cpu())

    def _draft(self, token):
        """Tokens and parents of a tree whose root is `token`, level by level."""
        tokens, parents, level = [token], [-1], [0]
        for width in WIDTHS:
            level = [(p, int(t)) for p in level for t in self.guess[tokens[p], :width]]
            parents += [p for p, _ in level]
            tokens += [t for _, t in level]
            level = list(range(len(tokens) - len(level), len(tokens)))
        return tokens, parents

    def step(self, names):
        """Draft, verify and keep for each of these requests; how many tokens each gained."""
        drafts = [self._draft(self.tokens[r][-1]) for r in names]
        step, tree_len, x = self._forward(names, [t for t, _ in drafts], [p for _, p in drafts])
        choice, at, paths = self._next(x), 0, []
        for r, (tokens, parents) in zip(names, drafts):
            path = [0]
            while True:
                want = choice[at + path[-1]]
                child = [i for i, p in enumerate(parents) if p == path[-1] and tokens[i] == want]
                if not child:
                    break
                path.append(child[0])
            self.tokens[r] += [tokens[i] for i in path[1:]] + [want]
            self.seen[r] += list(x[at:at + len(tokens)][path].float().cpu())
            at += len(tokens)
            paths.append(path)
        keep = np.full((len(names), max(map(len, paths))), -1)
        for r, path in enumerate(paths):
            keep[r, :len(path)] = path
        ctx = torch.empty(len(names), dtype=torch.int32, device=self.dev)
        pw.pw_kv_keep(self.attn, step, tree_len, self._i32(keep), self._i32([len(p) for p in paths]), ctx_out=ctx)
        for r, c in zip(names, ctx.tolist()):
            self.ctx[r] = c
            pw.pw_kv_trim(self.kv, r, -(-c // BLOCK))
        pw.pw_attn_check(self.attn)
        return [len(p) for p in paths]

    def fork(self, parent, child):
        """`child` goes on from where `parent` is; their blocks are shared but for the one that is written to next."""
        n = -(-self.ctx[parent] // BLOCK)
        pw.pw_kv_fork(self.kv, parent, child, n)
        self.row[child], self.ctx[child] = self.free_rows.pop(0), self.ctx[parent]
        self.tokens[child], self.seen[child] = list(self.tokens[parent]), list(self.seen[parent])
        row = self.table[self.row[child]]
        row.copy_(self.table[self.row[parent]])
        if self.ctx[child] % BLOCK:
            src, dst = pw.pw_kv_unshare(self.kv, child, n - 1)
            pw.pw_kv_copy(self.attn, self._i32([src]), self._i32([dst]))
            row[n - 1] = dst

    def release(self, request):
        pw.pw_kv_release(self.kv, request)
        row = self.row.pop(request)
        self.table[row] = -1
        self.free_rows.append(row)

    def compact(self):
        """The blocks in use lie side by side from block 0 on; how many moved."""
        src, dst = pw.pw_kv_compact(self.kv, pw.pw_kv_get_stats(self.kv)["used_blocks"])
        pw.pw_kv_copy(self.attn, self._i32(src), self._i32(dst), table=self.table)
        torch.cuda.synchronize()
        return len(src)

    def close(self):
        torch.cuda.synchronize()
        pw.pw_attn_destroy(self.attn)
        pw.pw_kv_destroy(self.kv)


def main(steps=4, seed=0):
    """Tokens of every request, their last hidden states, tokens gained by each verified tree, and blocks moved."""
    s = Server(max_requests=4, max_tokens=256, n_blocks=64, seed=seed)
    rng = np.random.default_rng(seed)
    for r, n in enumerate((37, 5, 90)):
        s.admit(r, rng.integers(0, VOCAB, n).tolist())
    gained = []
    for _ in range(steps):
        gained += s.step([0, 1, 2])
    s.fork(2, 3)
    s.tokens[3][-1] = (s.tokens[3][-1] + 1) % VOCAB  # another continuation
    for _ in range(steps):
        gained += s.step([3, 0, 2])
    s.release(0)
    moved = s.compact()
    for _ in range(steps):
        gained += s.step([1, 2, 3])
    s.close()
    return s.tokens, s.seen, gained, moved


if __name__ == "__main__":
    tokens, _, gained, moved = main()
    for r, t in tokens.items():
        print(f"request {r}: {len(t)} tokens")
    print(f"{sum(gained) / len(gained):.2f} tokens a verified tree; {moved} blocks moved by the compaction")
