"""Set-up of the tests with drafted trees: the paged-attention step of attn_helpers, with trees at the requests' ends."""
from __future__ import annotations

import numpy as np

from attn_helpers import UNIT, Step
from oracle import attn as oa


def random_tree(n, seed, back=None):
    """Parents of n nodes, each any earlier one of the last `back`, or -1."""
    rng = np.random.default_rng(seed)
    return [int(rng.integers(max(-1, i - back) if back else -1, i)) for i in range(n)]


def chain(n):
    return list(range(-1, n - 1))


class TreeStep(Step):
    """trees: parents of every request's nodes, which are its last tokens (some of them in the cache already)."""

    def __init__(self, ctx, new, trees, **kw):
        super().__init__(ctx, new, **kw)
        t, pw = self.torch, self.pw
        pw.pw_attn_destroy(self.attn)
        self.attn = pw.pw_attn_create(pw.pw_attn_desc(
            L=1, n_heads=self.Hq, n_kv_heads=self.Hkv, head_dim=self.D,
            dtype=pw.PW_BF16 if self.dtype == "bf16" else pw.PW_FP16, n_blocks=self.n_blocks, block_tokens=self.bt,
            max_requests=self.R, max_tokens=self.N, max_shared_tokens=self.N if self.groups is not None else 0,
            n_plans=kw.get("n_plans", 1), device=0, max_tree_tokens=self.N))
        pw.pw_attn_bind(self.attn, 0, *self.kv)
        self.tree_pos = t.full((self.N,), -7, dtype=t.int32, device="cuda")
        self.set_trees(trees)

    def set_trees(self, trees):
        t = self.torch
        self.trees = [list(x) for x in trees]
        width = max([len(x) for x in self.trees] + [1])
        flat = np.full((self.R, width), 99, dtype=np.int32)  # (behind a tree: not read)
        for r, x in enumerate(self.trees):
            flat[r, :len(x)] = x
        tree_len, parent = np.array([len(x) for x in self.trees], dtype=np.int32), flat
        if hasattr(self, "tree_len") and self.parent.shape == parent.shape:  # a captured call's tensors stay where they are
            self.tree_len.copy_(t.as_tensor(tree_len))
            self.parent.copy_(t.as_tensor(parent))
        else:
            self.tree_len, self.parent = t.as_tensor(tree_len).cuda(), t.as_tensor(parent).cuda()

    def plan(self, window=0, plan=0, stream=None):
        self.pw.pw_attn_plan_tree(self.attn, plan, self.step, self.tree_len, self.parent, pos=self.tree_pos, window=window,
                                  stream=stream)

    def forward(self, window=0, softcap=0.0, slopes=None, scale=None, check=True):
        t = self.torch
        keep = None if slopes is None else t.as_tensor(np.asarray(slopes, dtype=np.float32)).cuda()
        buf = t.full((self.N, self.Hq, 2, self.D), float("nan"), dtype=self.dt, device="cuda")
        o, lse = buf[:, :, 0], t.full((self.N, self.Hq), float("nan"), device="cuda")
        t.cuda.synchronize()
        self.plan(window)
        self.pw.pw_attn_forward(self.attn, 0, 0, self.q, o, lse=lse, scale=scale, softcap=softcap, slopes=keep)
        if check:
            self.pw.pw_attn_check(self.attn)
        else:
            t.cuda.synchronize()
        assert bool(t.isnan(buf[:, :, 1].float()).all()), "wrote beside o"
        return o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def expect(self, window=0, softcap=0.0, slopes=None, scale=None):
        where = oa.tree_rows(self.ctx, self.new, [len(x) for x in self.trees], self.trees, window)
        f = lambda x: x.float().cpu().numpy()  # noqa: E731
        n = len(where)
        with np.errstate(invalid="ignore"):
            out = oa.tree_attention(f(self.q)[:n], f(self.kv[0]), f(self.kv[1]), self.maps()[0], where, self.bt,
                                    self.D ** -0.5 if scale is None else scale, softcap, slopes, self.rows)
        return (*out, where)

    def compare(self, **kw):
        """The step's o, lse and positions against the oracle, with Step.compare's tolerances."""
        got, got_lse = self.forward(**kw)
        o, lse, absum, xmax, where = self.expect(**kw)
        n = len(where)
        self.near(got[:n], o, absum, max([len(w[2]) for w in where] + [1]))
        err = np.abs(got_lse[:n] - lse)
        lim = 2.0 ** -23 * (self.D + 16) * (4.0 + xmax)
        assert (err <= lim).all(), float((err / lim).max())
        assert not got[n:].any() and np.isneginf(got_lse[n:]).all()  # padding rows
        assert self.tree_pos.tolist() == [w[1] for w in where] + [-1] * (self.N - n)

    def near(self, got, o, absum, keys):
        u, v = UNIT[self.dtype], self.kv[1].float().cpu().numpy()
        vmax = float(np.nanmax(np.abs(v), initial=0.0, where=np.isfinite(v)))
        bad = ~(np.abs(got - o) <= u * (np.abs(o) + absum) + 1e-4 * absum + keys * 2.0 ** -25 * vmax + 1e-30)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(np.abs(got - o).max()))
