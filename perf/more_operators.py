"""Cases of the operators around the paged cache that drafting and page keeping need: norms and rotation with the
cache write, plans and attention of drafted trees, keeping an accepted path, and copying blocks.

``run`` computes a case with elementary torch operations in 32 bits (angles in 64), or, where ``own`` is true, with the
framework's calls.  ``exact`` restates each operator in 64 bits."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(op, **kw):
    c = dict(op=op, R=1, nodes=1, depth=1, held=0, chunks=0, chunk_max=0, ctx_min=0, ctx_max=0, bt=16, Hq=32, Hkv=8, D=128,
             L=1, dtype="bf16", rot=128, interleaved=False, axes=1, norm=False, theta=10000.0, window=0, softcap=0.0,
             alibi=False, lse=False, pairs=0, mix=1)
    c.update(kw)
    return c


def listed():
    return [
        # one layer's rotation and cache write for a few users' next tokens, far into their contexts: latency
        _case("rope", name="rope-decode-5", R=5, ctx_min=90000, ctx_max=131071, rot=64, interleaved=True, bt=64, mix=41),
        # the same of a long prompt, with norms of queries and keys: memory
        _case("rope", name="rope-prompt-8205", R=3, chunks=3, chunk_max=8205, ctx_max=700, norm=True, theta=500000.0, mix=42),
        # image tokens with positions in time, height and width, unshared heads of 96
        _case("rope", name="rope-images-5003", R=4, chunks=4, chunk_max=5003, ctx_max=300, Hq=16, Hkv=16, D=96, rot=96, axes=3,
              dtype="fp16", bt=32, mix=43),
        # the plan of a single user's draft of 24 tokens
        _case("plan", name="plan-1x24", nodes=24, depth=5, ctx_min=2017, ctx_max=2017, mix=44),
        # the plan of a server's drafts, up to 64 tokens for each of 96 requests
        _case("plan", name="plan-96x64", R=96, nodes=64, depth=6, ctx_min=16, ctx_max=8192, mix=45),
        # one layer's attention of the single user's draft: latency
        _case("tree", name="tree-1x24", nodes=24, depth=5, ctx_min=2017, ctx_max=2017, mix=46),
        # one layer's attention of a batch of drafts: memory and tensor cores alike
        _case("tree", name="tree-32x64", R=32, nodes=64, depth=6, ctx_min=256, ctx_max=8192, mix=47),
        # drafts of odd sizes in one step with prompt chunks, half of whose nodes were written by an earlier step
        _case("tree", name="tree-mixed-13", R=13, nodes=31, depth=5, held=2, chunks=4, chunk_max=1501, ctx_min=30, ctx_max=3001,
              Hq=16, Hkv=4, D=96, dtype="fp16", softcap=30.0, lse=True, bt=32, mix=48),
        # a single user's accepted tokens, moved in all layers of a model: latency
        _case("keep", name="keep-1", nodes=24, depth=4, ctx_min=300, ctx_max=300, L=24, mix=49),
        # a server's
        _case("keep", name="keep-96", R=96, nodes=64, depth=6, ctx_min=16, ctx_max=700, L=16, mix=50),
        # the last blocks of three requests, copied because a fork is about to write to them
        _case("copy", name="copy-3", R=3, pairs=3, ctx_min=40, ctx_max=300, L=24, mix=51),
        # a cache compacted, for its last third to be given back
        _case("copy", name="copy-700", R=64, pairs=700, ctx_min=200, ctx_max=900, L=12, Hkv=8, mix=52),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "plan", "tree", "tree", "tree", "keep", "copy"])
    Hq, Hkv = rng.choice([(32, 8), (16, 16), (32, 4), (8, 1), (24, 8), (28, 4), (16, 2), (8, 8)])
    D = rng.choice([64, 72, 80, 96, 128, 128])
    c = _case(op, Hq=Hq, Hkv=Hkv, D=D, rot=D, dtype=rng.choice(["bf16", "fp16"]), bt=rng.choice([16, 16, 32, 64, 128]),
              mix=rng.randrange(1 << 30))
    if op == "rope":
        R = _log(rng, 1, 64)
        c.update(R=R, ctx_max=_log(rng, 16, 100000 // R), rot=rng.choice([D, D, D // 16 * 8]), interleaved=rng.random() < 0.4,
                 axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.6, theta=rng.choice([1e4, 5e5, 1e6]))
        if rng.random() < 0.6:
            c.update(chunks=R, chunk_max=R + _log(rng, 1, 8000))
        return c
    R = _log(rng, 1, 48)
    c.update(R=R, nodes=_log(rng, 1, 128), depth=rng.randrange(1, 9))
    if op == "keep":
        c.update(ctx_max=_log(rng, 16, 700), L=rng.randrange(1, 17))
    elif op == "copy":
        c.update(ctx_min=10, ctx_max=_log(rng, 64, 700), L=rng.randrange(1, 13), pairs=_log(rng, 1, 500))
    else:
        # at most half of tree-32x64's rows times keys
        top = _log(rng, 64, min(16384, 8000000 // (R * c["nodes"])))
        c.update(ctx_min=min(top, rng.randrange(0, 200)), ctx_max=top, window=rng.choice([0, 0, 0, rng.randrange(3, 2000)]),
                 held=rng.choice([0, 0, 1, 2]), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.25,
                 lse=rng.random() < 0.25)
        if R > 2 and rng.random() < 0.3:
            c.update(chunks=rng.randrange(1, R), chunk_max=R + _log(rng, 8, 700), ctx_max=min(top, 2000), ctx_min=0)
    return c


# ------------------------------------------------------------------ what a case is, apart from its inputs
def _cdiv(a, b):
    return -(-a // b)


class Shape:
    """Lengths of a case's requests.  The tree of request r is its last nodes[r] keys, from position start[r], in levels
    of levels[r] nodes, of which the first levels may lie in the cache from an earlier step.  The first `chunks` requests have
    new tokens without a tree."""

    def __init__(self, case):
        rng = np.random.default_rng(case["mix"])
        R, chunks = case["R"], case["chunks"]
        self.any_tree = case["op"] == "plan"
        self.start = rng.integers(case["ctx_min"], case["ctx_max"] + 1, size=R)
        self.start[-1] = case["ctx_max"]
        self.nodes = rng.integers((case["nodes"] + 1) // 2, case["nodes"] + 1, size=R)
        self.nodes[-1] = case["nodes"]
        self.levels, held = [], np.zeros(R, dtype=np.int64)
        for r in range(R):
            n = int(self.nodes[r])
            d = min(case["depth"], (n + 1) // 2)
            size = np.full(d, max(1, (n - d) // d))
            size[0] = n - size[1:].sum()  # d or more: an accepted path moves to places that it does not come from
            self.levels.append(size)
            held[r] = size[:min(case["held"], d - 1)].sum()
        self.new = self.nodes - held
        if case["op"] == "rope":
            self.new[:] = 1
            self.nodes[:] = held[:] = 0
        if chunks:  # new tokens without a tree, chunk_max in all
            w = rng.exponential(size=chunks) ** 2
            n = 1 + np.floor(w / w.sum() * (case["chunk_max"] - chunks)).astype(np.int64)
            n[0] += case["chunk_max"] - n.sum()
            self.new[:chunks] = n
            self.nodes[:chunks] = held[:chunks] = 0
        self.ctx = self.start + held
        self.kv = self.ctx + self.new
        self.N = int(self.new.sum())
        self.q_start = np.concatenate([[0], np.cumsum(self.new)])
        self.row = np.repeat(np.arange(R), self.new)                       # request of a row
        self.at = np.arange(self.N) - self.q_start[self.row] + self.ctx[self.row]  # its place in the cache
        # accepted path of a request: the first node of each of its first levels
        self.n_keep = np.array([int(rng.integers(0, len(s) + 1)) for s in self.levels])
        self.n_keep[-1] = len(self.levels[-1])
        self.path = [np.concatenate([[0], np.cumsum(s)[:-1]]) for s in self.levels]

    def depths(self, r):
        return np.repeat(np.arange(len(self.levels[r])), self.levels[r])

    def parents(self, seed):
        """Parent of every node, request by request [R][most nodes]: one of the level before, in ascending order, and of the first
        node of a level the first one; -1 for the first level.  For a plan alone, which takes the same time for any
        tree, any earlier node."""
        rng = np.random.default_rng(seed)
        out = np.full((len(self.levels), max(1, int(self.nodes.max()))), -1, dtype=np.int32)
        if self.any_tree:
            return rng.integers(-1, np.broadcast_to(np.arange(out.shape[1]), out.shape)).astype(np.int32)
        for r, sizes in enumerate(self.levels):
            if self.nodes[r] == 0:
                continue
            first = np.concatenate([[0], np.cumsum(sizes)])
            for i in range(1, len(sizes)):
                p = np.sort(rng.integers(0, sizes[i - 1], size=sizes[i]))
                p[0] = 0
                out[r, first[i]:first[i + 1]] = first[i - 1] + p
        return out


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(DEV)


def _inv_freq(case):
    return case["theta"] ** (-np.arange(0, case["rot"], 2) / case["rot"])


def _axis(case):
    """Axis of each pair: a quarter of them follow time, the rest height and width."""
    n = case["rot"] // 2
    if case["axes"] == 1:
        return np.zeros(n, dtype=np.int32)
    t = n // 4
    h = (n - t) // 2
    return np.repeat(np.arange(3), [t, h, n - t - h]).astype(np.int32)


def _pairs(case):
    i = np.arange(case["rot"] // 2)
    return (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)


def prepare(case, seed):
    """The paged cache, the step's lengths and new rows; beside them the attention handle, its bound caches, the rotation's
    tables and the plan that a program makes once for a step's layers."""
    s = Shape(case)
    R, bt, D, L, Hq, Hkv, N = case["R"], case["bt"], case["D"], case["L"], case["Hq"], case["Hkv"], s.N
    op, dt = case["op"], DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    pages = _cdiv(s.kv, bt)
    width = int(pages.max())
    used = int(pages.sum())
    n_blocks = used + 3 + (case["pairs"] if op == "copy" else 0)
    perm = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((R, width), -1, dtype=np.int32)
    table[np.arange(width)[None] < pages[:, None]] = perm[:used]
    slot = table[s.row, s.at // bt].astype(np.int64) * bt + s.at % bt
    st = dict(case=case, R=R, N=N, n_blocks=n_blocks, max_new=int(s.new.max()), max_kv=int(s.kv.max()), table=_i32(table),
              ctx_len=_i32(s.ctx), new_len=_i32(s.new), kv_len=_i32(s.kv), q_start=_i32(s.q_start),
              slot=torch.as_tensor(slot).to(DEV), pos=_i32(s.at), row=torch.as_tensor(s.row).to(DEV),
              tree_len=_i32(s.nodes), parent=_i32(s.parents(seed)), tree_pos=torch.zeros(N, dtype=torch.int32, device=DEV))
    if op != "plan":
        st["cache"] = torch.randn((L, 2, n_blocks, bt, Hkv, D), dtype=dt, device=DEV, generator=g)
    if op == "rope":  # q, k and v as a fused projection leaves them: slices of one row
        qkv = torch.randn(N, Hq + 2 * Hkv, D, dtype=dt, device=DEV, generator=g)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["q_out"] = torch.empty(N, Hq, D, dtype=dt, device=DEV)
        st["q_gain"] = st["k_gain"] = None
        if case["norm"]:
            gains = 1 + 0.2 * torch.randn(2, D, device=DEV, generator=g)
            st["q_gain"], st["k_gain"] = gains[0], gains[1]
        st["axes_pos"] = None
        if case["axes"] == 3:  # a frame's time, and places in a grid that begins there
            p = s.at[None] + np.stack([np.zeros(N, dtype=np.int64), rng.integers(0, 64, N), rng.integers(0, 64, N)])
            st["axes_pos"] = _i32(p)
        st["inv_freq"] = torch.as_tensor(_inv_freq(case)).to(DEV)
        st["axis"] = torch.as_tensor(_axis(case)).long().to(DEV)
        st["first"], st["second"] = (torch.as_tensor(i).to(DEV) for i in _pairs(case))
    if op == "tree":
        st["q"] = torch.randn(N, Hq, D, device=DEV, generator=g).mul_(1.5).to(dt)
        st["o"] = torch.empty(N, Hq, D, dtype=dt, device=DEV)
        st["lse"] = torch.empty(N, Hq, device=DEV) if case["lse"] else None
        st["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if case["alibi"] else None
    if op == "keep":
        keep = np.full((R, max(len(p) for p in s.path)), -1, dtype=np.int32)
        for r in range(R):
            keep[r, :s.n_keep[r]] = s.path[r][:s.n_keep[r]]
        st["keep"], st["n_keep"] = _i32(keep), _i32(s.n_keep)
        st["ctx_out"] = torch.zeros(R, dtype=torch.int32, device=DEV)
    if op == "copy":
        n = min(case["pairs"], used)
        st["src"], st["dst"] = _i32(rng.choice(perm[:used], size=n, replace=False)), _i32(perm[used:used + n])
    _prepare_own(st)
    return st


class _Handle:
    """An attention handle, released with the state that holds it."""

    def __init__(self, pw, desc):
        self.pw, self.h = pw, pw.pw_attn_create(desc)

    def __del__(self):
        self.pw.pw_attn_destroy(self.h)


def _prepare_own(st):
    if not own:
        return
    import any_precision_bit_gb300 as pw
    c = st["case"]
    st["pw"] = pw
    st["handle"] = _Handle(pw, pw.pw_attn_desc(
        L=c["L"], n_heads=c["Hq"], n_kv_heads=c["Hkv"], head_dim=c["D"],
        dtype=pw.PW_BF16 if c["dtype"] == "bf16" else pw.PW_FP16, n_blocks=st["n_blocks"], block_tokens=c["bt"],
        max_requests=c["R"], max_tokens=st["N"], max_shared_tokens=0, max_tree_tokens=st["N"], n_plans=1, device=0))
    h = st["handle"].h
    st["step"] = pw.pw_make_step(st["ctx_len"], st["new_len"], st["table"], st["q_start"], st["kv_len"], st["slot"],
                                 st["pos"], max_new=st["max_new"])
    if "cache" in st:
        for layer in range(c["L"]):
            pw.pw_attn_bind(h, layer, st["cache"][layer, 0], st["cache"][layer, 1])
    if c["op"] == "rope":
        pw.pw_attn_set_rope(h, 0, _inv_freq(c), axis=_axis(c), n_axes=c["axes"], interleaved=c["interleaved"],
                            q_gain=st["q_gain"], k_gain=st["k_gain"], eps=1e-6)
    if c["op"] == "tree":
        pw.pw_attn_plan_tree(h, 0, st["step"], st["tree_len"], st["parent"], pos=st["tree_pos"], window=c["window"],
                             stream=torch.cuda.current_stream())


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _plain_rope, "plan": _plain_plan, "tree": _plain_tree, "keep": _plain_keep, "copy": _plain_copy}[op](state)


def _own(st, op):
    pw, h, c, stream = st["pw"], st["handle"].h, st["case"], torch.cuda.current_stream()
    if op == "rope":
        pw.pw_attn_rope_append(h, 0, st["step"], st["q"], st["q_out"], st["k"], st["v"], pos=st["axes_pos"], stream=stream)
        return {"q": st["q_out"], "cache": st["cache"]}
    if op == "plan":
        pw.pw_attn_plan_tree(h, 0, st["step"], st["tree_len"], st["parent"], pos=st["tree_pos"], window=c["window"],
                             stream=stream)
        return {"pos": st["tree_pos"]}
    if op == "tree":
        pw.pw_attn_forward(h, 0, 0, st["q"], st["o"], lse=st["lse"], softcap=c["softcap"], slopes=st["slopes"], stream=stream)
        return {"o": st["o"]} if st["lse"] is None else {"o": st["o"], "lse": st["lse"]}
    if op == "keep":
        pw.pw_kv_keep(h, st["step"], st["tree_len"], st["keep"], st["n_keep"], ctx_out=st["ctx_out"], stream=stream)
        return {"cache": st["cache"], "ctx_len": st["ctx_out"]}
    pw.pw_kv_copy(h, st["src"], st["dst"], table=st["table"], stream=stream)
    return {"cache": st["cache"], "table": st["table"]}


# ------------------------------------------------------------------ plain forms
def _plain_rope(st):
    c = st["case"]
    n_blocks, bt, Hkv, D = st["cache"].shape[2:]
    pos = st["axes_pos"] if st["axes_pos"] is not None else st["pos"][None]
    angle = pos.double()[st["axis"]].T * st["inv_freq"]  # [N][rot / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, gain):
        y = x.float()
        if gain is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * gain
        a, b = y[..., st["first"]], y[..., st["second"]]
        out = y.clone()
        out[..., st["first"]] = a * cos - b * sin
        out[..., st["second"]] = a * sin + b * cos
        return out.to(x.dtype)

    st["cache"][0, 0].view(n_blocks * bt, Hkv, D)[st["slot"]] = turned(st["k"], st["k_gain"])
    st["cache"][0, 1].view(n_blocks * bt, Hkv, D)[st["slot"]] = st["v"]
    st["q_out"].copy_(turned(st["q"], st["q_gain"]))
    return {"q": st["q_out"], "cache": st["cache"]}


def _squared(seen):
    return torch.matmul(seen, seen).clamp_(max=1.0)


def _ancestors(st):
    """[R][P][P]: node j is i or one of its ancestors (paths of up to 256 steps); and depths [R][P]."""
    parent = st["parent"].long()
    P = parent.shape[1]
    node = torch.arange(P, device=DEV)
    seen = ((parent[:, :, None] == node) | (node[:, None] == node)).float()
    seen = _squared(_squared(_squared(_squared(_squared(_squared(_squared(_squared(seen))))))))
    return seen, seen.sum(-1).long() - 1


def _positions(st, depth):
    """Node of every row (-1: none), the tree's start, and the row's position."""
    row = st["row"]
    start = (st["kv_len"] - st["tree_len"])[row].long()
    at = st["pos"].long()
    node = torch.where(at >= start, at - start, torch.full_like(at, -1))
    return node, start, torch.where(node >= 0, start + depth[row, node.clamp(min=0)], at)


def _plain_plan(st):
    _, depth = _ancestors(st)
    return {"pos": _positions(st, depth)[2].int()}


def _plain_tree(st):
    c = st["case"]
    R, Hq, Hkv, D, Tm, Lm = st["R"], c["Hq"], c["Hkv"], c["D"], st["max_new"], st["max_kv"]
    G = Hq // Hkv
    seen, depth = _ancestors(st)
    node, start, pos = _positions(st, depth)
    # keys and values of every request, padded: [R, Hkv, L, D]
    blocks = st["table"].long().clamp(min=0)
    k = st["cache"][0, 0][blocks].flatten(1, 2)[:, :Lm].permute(0, 2, 1, 3).float()
    v = st["cache"][0, 1][blocks].flatten(1, 2)[:, :Lm].permute(0, 2, 1, 3).float()
    # queries, padded: [R, Hkv, Tm * G, D]
    first = st["q_start"][:-1].long()
    i = torch.arange(Tm, device=DEV)
    t = (first[:, None] + i).clamp(max=st["N"] - 1)  # [R, Tm]
    q = st["q"][t].float().view(R, Tm, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, Tm * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(R, Hkv, Tm, G, Lm)
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    # positions of keys: those of a tree lie at their depths
    j = torch.arange(Lm, device=DEV)
    begin = (st["kv_len"] - st["tree_len"]).long()[:, None]
    in_tree = (j >= begin) & (j < st["kv_len"].long()[:, None])  # [R, Lm]
    knode = (j - begin).clamp(0, depth.shape[1] - 1)
    key_pos = torch.where(in_tree, begin + torch.gather(depth, 1, knode), j.expand(R, Lm))
    away = pos[t][:, :, None] - key_pos[:, None]  # [R, Tm, Lm]
    if st["slopes"] is not None:
        x = x - st["slopes"].view(1, Hkv, 1, G, 1) * away.abs().float()[:, None, :, None, :]
    own_nodes = torch.gather(seen, 1, node[t].clamp(min=0)[:, :, None].expand(R, Tm, seen.shape[2]))  # [R, Tm, P]
    above = torch.gather(own_nodes, 2, knode[:, None].expand(R, Tm, Lm)) > 0
    see = torch.where(in_tree[:, None] & (node[t] >= 0)[:, :, None], above, j <= st["pos"].long()[t][:, :, None])
    if c["window"]:
        see = see & (away < c["window"])
    x = torch.where(see[:, None, :, None, :], x, torch.full_like(x[:1, :1, :1, :1, :1], -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    del x
    s = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hkv, Tm * G, Lm), v).view(R, Hkv, Tm, G, D) / s
    tt = torch.arange(st["N"], device=DEV) - first[st["row"]]
    out = {"o": o.permute(0, 2, 1, 3, 4)[st["row"], tt].reshape(st["N"], Hq, D).to(st["q"].dtype)}
    if st["lse"] is not None:
        out["lse"] = (m + torch.log(s))[..., 0].permute(0, 2, 1, 3)[st["row"], tt].reshape(st["N"], Hq)
    return out


def _plain_keep(st):
    L, _, n_blocks, bt, Hkv, D = st["cache"].shape
    start = (st["kv_len"] - st["tree_len"]).long()
    i = torch.arange(st["keep"].shape[1], device=DEV)
    some = i < st["n_keep"][:, None]
    r = torch.arange(st["R"], device=DEV)[:, None].expand_as(some)[some]
    to, at = (start[:, None] + i)[some], (start[:, None] + st["keep"].long())[some]
    table = st["table"].long()
    flat = st["cache"].view(L, 2, n_blocks * bt, Hkv, D)
    moved = flat[:, :, table[r, at // bt] * bt + at % bt]
    flat[:, :, table[r, to // bt] * bt + to % bt] = moved
    return {"cache": st["cache"], "ctx_len": (start + st["n_keep"].long()).int()}


def _plain_copy(st):
    src, dst, table = st["src"].long(), st["dst"].long(), st["table"]
    st["cache"][:, :, dst] = st["cache"][:, :, src]
    renamed = torch.arange(st["n_blocks"], device=DEV, dtype=torch.int32)
    renamed[src] = st["dst"]
    st["table"].copy_(torch.where(table >= 0, renamed[table.long().clamp(min=0)], table))
    return {"cache": st["cache"], "table": st["table"]}


# ------------------------------------------------------------------ costs
def work(case):
    s = Shape(case)
    R, bt, D, Hq, Hkv, N, L = case["R"], case["bt"], case["D"], case["Hq"], case["Hkv"], s.N, case["L"]
    token = Hkv * D * 2  # bytes of a token's keys, or values, in one layer
    if case["op"] == "rope":
        return {"bytes": 2 * 2 * N * (Hq + 2 * Hkv) * D + (8 + 4 * case["axes"]) * N, "flops": 6 * N * (Hq + Hkv) * D}
    if case["op"] == "plan":
        return {"bytes": 16 * R + 4 * int(s.nodes.sum()) + 4 * N, "flops": 0}
    if case["op"] == "keep":
        moved = sum(int((s.path[r][:s.n_keep[r]] != np.arange(s.n_keep[r])).sum()) for r in range(R))
        return {"bytes": 2 * 2 * moved * L * token + 4 * int(s.n_keep.sum()) + 16 * R, "flops": 0}
    if case["op"] == "copy":
        n = min(case["pairs"], int(_cdiv(s.kv, bt).sum()))
        return {"bytes": 2 * 2 * n * L * bt * token + 8 * n + 8 * int(_cdiv(s.kv, bt).sum()), "flops": 0}
    lo, see = _visible(case, s)
    span = np.full(R, np.iinfo(np.int64).max)
    np.minimum.at(span, s.row, lo)
    keys = int(np.maximum(0, s.kv - span).sum())
    return {"bytes": 2 * keys * token + 2 * N * Hq * D * 2 + 4 * _cdiv(keys, bt) + (4 * N * Hq if case["lse"] else 0),
            "flops": 4 * D * Hq * int(see.sum())}


def _visible(case, s):
    """Position of the first key and number of keys that every row sees (a node at depth d sees d ancestors)."""
    lo, see = np.zeros(s.N, dtype=np.int64), np.zeros(s.N, dtype=np.int64)
    for r in range(case["R"]):
        rows = slice(s.q_start[r], s.q_start[r + 1])
        pos = s.at[rows].copy()
        if s.nodes[r]:
            pos = s.start[r] + s.depths(r)[pos - s.start[r]]
        lo[rows] = np.maximum(0, pos - case["window"] + 1) if case["window"] else 0
        see[rows] = pos + 1 - lo[rows]
    return lo, see


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st, s = prepare(case, seed), Shape(case)
    bt, D, Hq, Hkv = case["bt"], case["D"], case["Hq"], case["Hkv"]
    if case["op"] == "plan":  # whole numbers: the plain form's are exact
        return None
    if case["op"] == "rope":
        freq, axis = _inv_freq(case), _axis(case)
        pos = np.stack([s.at] * 3) if st["axes_pos"] is None else st["axes_pos"].cpu().numpy()
        turn = torch.as_tensor(np.exp(1j * (pos[axis].T.astype(np.float64) * freq[None]))).to(DEV)[:, None]
        n = case["rot"] // 2

        def turned(x, gain):
            x = x.double()
            if gain is not None:
                x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * gain.double()
            head = x[..., :2 * n].unflatten(-1, (n, 2) if case["interleaved"] else (2, n))
            pair = -1 if case["interleaved"] else -2
            z = torch.complex(head.select(pair, 0), head.select(pair, 1)) * turn
            return torch.cat([torch.stack([z.real, z.imag], pair).flatten(-2), x[..., 2 * n:]], -1)

        cache = st["cache"].double()
        cache[0, 0][st["slot"] // bt, st["slot"] % bt] = turned(st["k"], st["k_gain"])
        cache[0, 1][st["slot"] // bt, st["slot"] % bt] = st["v"].double()
        return {"q": turned(st["q"], st["q_gain"]), "cache": cache}
    if case["op"] == "keep":
        cache, table = st["cache"].clone(), st["table"].cpu().numpy()
        for r in range(case["R"]):
            for i in range(s.n_keep[r]):
                a, b = int(s.start[r] + s.path[r][i]), int(s.start[r] + i)
                cache[:, :, table[r, b // bt], b % bt] = st["cache"][:, :, table[r, a // bt], a % bt]
        return {"cache": cache.double(), "ctx_len": None}
    if case["op"] == "copy":
        cache = st["cache"].clone()
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            cache[:, :, b] = st["cache"][:, :, a]
        return {"cache": cache.double(), "table": None}
    parents = s.parents(seed)
    G = Hq // Hkv
    o = torch.zeros(s.N, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s.N, Hq, dtype=torch.float64, device=DEV)
    head = torch.arange(1, Hq + 1, dtype=torch.float64, device=DEV)
    for r in range(case["R"]):
        b, e, n, start = int(s.q_start[r]), int(s.q_start[r + 1]), int(s.kv[r]), int(s.start[r])
        place = np.arange(n)  # the keys' positions
        see = place[None] <= s.at[b:e, None]
        if s.nodes[r]:
            place = np.concatenate([place[:start], start + s.depths(r)])
            see = see & (place < start)[None]
            for t in range(b, e):
                i = int(s.at[t]) - start
                while i >= 0:
                    see[t - b, start + i] = True
                    i = int(parents[r, i])
            see[:, :start] = True
        away = place[s.at[b:e]][:, None] - place[None]
        if case["window"]:
            see = see & (away < case["window"])
        hide = torch.as_tensor(~see).to(DEV)
        far = torch.as_tensor(np.abs(away)).to(DEV).double()
        blocks = st["table"][r, :_cdiv(n, bt)].long()
        for h in range(Hkv):
            K = st["cache"][0, 0][blocks][:, :, h].reshape(-1, D)[:n].double()
            V = st["cache"][0, 1][blocks][:, :, h].reshape(-1, D)[:n].double()
            a = torch.einsum("tgd,ld->gtl", st["q"][b:e, h * G:(h + 1) * G].double(), K) / math.sqrt(D)
            if case["softcap"]:
                a = case["softcap"] * torch.tanh(a / case["softcap"])
            if case["alibi"]:
                slope = torch.exp2(-8.0 * head[h * G:(h + 1) * G] / Hq).float().double()
                a = a - slope[:, None, None] * far
            a = a.masked_fill(hide, -math.inf)
            z = torch.logsumexp(a, -1, keepdim=True)
            o[b:e, h * G:(h + 1) * G] = torch.matmul(torch.exp(a - z), V).transpose(0, 1)
            lse[b:e, h * G:(h + 1) * G] = z[..., 0].T
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
