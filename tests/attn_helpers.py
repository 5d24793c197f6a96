"""Set-up of the paged-attention tests: a step over a cache whose unwritten slots hold NaN, run
through the C ABI and compared with the float64 oracle."""
from __future__ import annotations

import numpy as np

from oracle import attn as oa

UNIT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}  # largest relative error of one rounding to nearest


class Step:
    def __init__(self, ctx, new, Hq=4, Hkv=2, D=64, bt=16, dtype="bf16", seed=0, layout="nhd", pad=0, rows=None,
                 prefix=0, group_start=None, spare_ids=0, n_plans=1, qscale=1.5):
        import torch

        import any_precision_bit_gb300 as pw
        self.torch, self.pw = torch, pw
        self.ctx, self.new = [int(c) for c in ctx], [int(n) for n in new]
        self.Hq, self.Hkv, self.D, self.bt, self.dtype = Hq, Hkv, D, bt, dtype
        dt = self.dt = {"bf16": torch.bfloat16, "fp16": torch.float16}[dtype]
        R, N = len(ctx), sum(new) + pad
        self.R, self.N, self.rows = R, N, rows
        rng = np.random.default_rng(seed)
        pages = [-(-(c + n) // bt) for c, n in zip(ctx, new)]
        held = [-(-c // bt) for c in ctx]
        n_rows = R if rows is None else max(rows) + 1
        self.n_blocks = nb = sum(pages) + 3
        perm = rng.permutation(nb)
        table = -np.ones((n_rows, max(max(pages), 1) + 1), dtype=np.int32)
        at = 0
        starts = list(range(R + 1)) if group_start is None else group_start
        lens = [prefix] * (len(starts) - 1) if np.isscalar(prefix) else list(prefix)
        first = {}
        for g in range(len(starts) - 1):
            for r in range(starts[g], starts[g + 1]):
                first[r] = (starts[g], lens[g] // bt)
        for r in range(R):
            row = r if rows is None else rows[r]
            lead, common = first[r]
            for p in range(held[r]):
                if lead != r and p < common:
                    table[row, p] = table[lead if rows is None else rows[lead], p]
                else:
                    table[row, p] = perm[at]
                    at += 1
        n_new = sum(p - h for p, h in zip(pages, held))
        ids = perm[at:at + n_new + spare_ids].astype(np.int32)
        self.table0, self.ids = table, ids
        # caches: NaN but where a request has written
        shape = (nb, bt, Hkv, D) if layout == "nhd" else (nb, Hkv, bt, D)
        g = torch.Generator().manual_seed(seed)
        self.kv = []
        for _ in range(2):
            c = torch.full(shape, float("nan"), dtype=dt)
            view = c if layout == "nhd" else c.permute(0, 2, 1, 3)
            for r in range(R):
                row = r if rows is None else rows[r]
                for p in range(held[r]):
                    n = min(bt, self.ctx[r] - p * bt)
                    view[int(table[row, p]), :n] = torch.randn(n, Hkv, D, generator=g).to(dt)
            dev = c.cuda()
            self.kv.append(dev if layout == "nhd" else dev.permute(0, 2, 1, 3))
        # q, k, v: slices of one row, as a fused projection leaves them
        qkv = torch.randn(N, Hq + 2 * Hkv, D, generator=g)
        qkv[:, :Hq] *= qscale
        self.qkv = qkv.to(dt).cuda()
        self.q, self.k, self.v = self.qkv[:, :Hq], self.qkv[:, Hq:Hq + Hkv], self.qkv[:, Hq + Hkv:]
        i32 = lambda a: torch.as_tensor(np.asarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.table = i32(table)
        self.q_start, self.kv_len = i32(np.zeros(R + 1)), i32(np.zeros(R))
        self.slot = torch.full((N,), -7, dtype=torch.int64, device="cuda")
        self.pos = i32(np.full(N, -7))
        self.new_ids = i32(ids)
        self.groups = None if group_start is None else i32(group_start)
        self.shared = None if group_start is None else i32(lens)
        self.attn = pw.pw_attn_create(pw.pw_attn_desc(
            L=1, n_heads=Hq, n_kv_heads=Hkv, head_dim=D, dtype=pw.PW_BF16 if dtype == "bf16" else pw.PW_FP16,
            n_blocks=nb, block_tokens=bt, max_requests=R, max_tokens=N,
            max_shared_tokens=N if group_start is not None else 0, n_plans=n_plans, device=0))
        pw.pw_attn_bind(self.attn, 0, *self.kv)
        self.step = pw.pw_make_step(i32(ctx), i32(new), self.table, self.q_start, self.kv_len, self.slot, self.pos,
                                    max_new=max(new), rows=None if rows is None else i32(rows), groups=self.groups,
                                    shared_len=self.shared)

    def map_and_append(self):
        self.torch.cuda.synchronize()
        self.pw.pw_kv_map(self.attn, self.step, self.new_ids)
        self.pw.pw_attn_append(self.attn, 0, self.step, self.k, self.v)

    def maps(self):
        return oa.step_maps(self.ctx, self.new, self.bt, self.ids, self.table0, self.rows, self.N)

    def forward(self, window=0, doc_start=None, bidir_len=None, softcap=0.0, slopes=None, scale=None, plan=0):
        t = self.torch
        dev = lambda a, dt: None if a is None else t.as_tensor(np.asarray(a, dtype=dt)).cuda()  # noqa: E731
        keep = dev(doc_start, np.int32), dev(bidir_len, np.int32), dev(slopes, np.float32)
        buf = t.full((self.N, self.Hq, 2, self.D), float("nan"), dtype=self.dt, device="cuda")
        o, lse = buf[:, :, 0], t.full((self.N, self.Hq), float("nan"), device="cuda")
        t.cuda.synchronize()
        self.pw.pw_attn_plan(self.attn, plan, self.step, window=window, doc_start=keep[0], bidir_len=keep[1])
        self.pw.pw_attn_forward(self.attn, 0, plan, self.q, o, lse=lse, scale=scale, softcap=softcap, slopes=keep[2])
        self.pw.pw_attn_check(self.attn)
        assert bool(t.isnan(buf[:, :, 1].float()).all()), "wrote beside o"
        return o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)

    def expect(self, window=0, doc_start=None, bidir_len=None, softcap=0.0, slopes=None, scale=None):
        table = self.maps()[0]
        where = oa.bounds(self.ctx, self.new, window, doc_start, bidir_len)
        f = lambda x: x.float().cpu().numpy()  # noqa: E731
        n = len(where)
        with np.errstate(invalid="ignore"):
            o, lse, absum, xmax = oa.attention(f(self.q)[:n], f(self.kv[0]), f(self.kv[1]), table, where, self.bt,
                                               self.D ** -0.5 if scale is None else scale, softcap, slopes, self.rows)
        return o, lse, absum, xmax, where

    def compare(self, **kw):
        """The whole step's o and lse against the oracle.  o: one rounding of the result, one of each
        probability (either at most `unit` of what it rounds), probabilities that underflow in fp16, and
        1e-4 of the fp32 steps before; lse: fp32 products and sums of D terms."""
        got, got_lse = self.forward(**kw)
        o, lse, absum, xmax, where = self.expect(**kw)
        n, u = len(where), UNIT[self.dtype]
        keys = max([hi - lo for _, _, lo, hi in where] + [1])
        vmax = float(np.nanmax(np.abs(self.kv[1].float().cpu().numpy()), initial=0.0, where=~np.isnan(self.kv[1].float().cpu().numpy())))
        tol = u * (np.abs(o) + absum) + 1e-4 * absum + keys * 2.0 ** -25 * vmax
        bad = ~(np.abs(got[:n] - o) <= tol + 1e-30)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(np.abs(got[:n] - o).max()))
        empty = np.array([lo >= hi for _, _, lo, hi in where], dtype=bool)
        assert not got[:n][empty].any() and np.isneginf(got_lse[:n][empty]).all()
        err = np.abs(got_lse[:n][~empty] - lse[~empty])
        lim = 2.0 ** -23 * (self.D + 16) * (4.0 + xmax[~empty])
        assert (err <= lim).all(), float((err / lim).max())
        assert not got[n:].any() and np.isneginf(got_lse[n:]).all()  # padding rows

    def close(self):
        self.pw.pw_attn_destroy(self.attn)
