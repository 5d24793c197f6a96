"""Cases of the paged-attention operators: the step maps, the cache write, attention over the
paged cache and attention over a shared prefix.

``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is
true, with the framework's calls.  ``exact`` restates each operator in 64 bits."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _case(op, **kw):
    c = dict(op=op, R=1, new_total=1, ctx_min=0, ctx_max=0, bt=16, Hq=32, Hkv=8, D=128, dtype="bf16", window=0,
             softcap=0.0, alibi=False, docs=0, bidir=False, prefix=0, lse=False, mix=1)
    c.update(kw)
    return c


def listed():
    return [
        # the maps of one decode step of a busy server: one new token for each of 64 requests
        _case("map", name="map-decode-64", R=64, new_total=64, ctx_min=16, ctx_max=8192, mix=11),
        # the maps of a step that mixes prompt chunks with a few hundred short continuations
        _case("map", name="map-mixed-384", R=384, new_total=32768, ctx_min=0, ctx_max=16384, mix=12),
        # one layer's cache write of a decode step
        _case("append", name="append-decode-64", R=64, new_total=64, ctx_min=16, ctx_max=8192, mix=13),
        # one layer's cache write of a long prompt, one key/value head for each query head
        _case("append", name="append-prompt-8205", R=3, new_total=8205, ctx_min=0, ctx_max=700, Hq=16, Hkv=16, bt=32,
              mix=14),
        # a single user's decode step: latency is all that counts
        _case("attn", name="decode-1-short", R=1, new_total=1, ctx_min=517, ctx_max=517, mix=15),
        # an ordinary decode batch of ragged contexts, four query heads to a key/value head
        _case("attn", name="decode-64", R=64, new_total=64, ctx_min=256, ctx_max=8192, mix=16),
        # a decode batch with two draft tokens each, windowed and capped scores, unshared heads
        _case("attn", name="decode-160-window-cap", R=160, new_total=320, ctx_min=30, ctx_max=6000, Hq=16, Hkv=16,
              D=64, dtype="fp16", window=1024, softcap=30.0, bt=32, mix=17),
        # a few very long contexts with a distance bias: the keys of one request go to many SMs
        _case("attn", name="decode-3-long-bias", R=3, new_total=3, ctx_min=90001, ctx_max=131071, Hkv=4, alibi=True,
              bt=64, lse=True, mix=18),
        # a whole prompt: the tensor cores' case
        _case("attn", name="prompt-8192", R=1, new_total=8192, mix=19),
        # prompt chunks of packed documents behind cached contexts, capped scores, a two-way prefix
        _case("attn", name="chunks-docs-cap", R=5, new_total=5003, ctx_min=0, ctx_max=2111, Hq=16, Hkv=4, D=96,
              dtype="fp16", softcap=50.0, docs=4, bidir=True, mix=20),
        # requests answering from one long system prompt
        _case("shared", name="prefix-64", R=64, new_total=64, ctx_min=1, ctx_max=256, prefix=4096, mix=21),
        # the largest such batch
        _case("shared", name="prefix-256", R=256, new_total=256, ctx_min=1, ctx_max=640, prefix=16384, mix=22),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "append", "attn", "attn", "attn", "shared"])
    Hq, Hkv = rng.choice([(32, 8), (16, 16), (32, 4), (8, 1), (24, 8), (28, 4), (16, 2), (8, 8)])
    c = _case(op, Hq=Hq, Hkv=Hkv, D=rng.choice([64, 80, 96, 128, 128]), dtype=rng.choice(["bf16", "fp16"]),
              bt=rng.choice([16, 16, 32, 64, 128]), mix=rng.randrange(1 << 30))
    if op == "map":
        R = _log(rng, 1, 512)
        c.update(R=R, new_total=R if rng.random() < 0.5 else R + _log(rng, 1, 32000),
                 ctx_max=_log(rng, 16, 16384))
    elif op == "append":
        R = _log(rng, 1, 64)
        c.update(R=R, new_total=R + (0 if rng.random() < 0.4 else _log(rng, 1, 8000)), ctx_max=_log(rng, 16, 4096))
    elif op == "shared":
        R = _log(rng, 2, 256)
        c.update(R=R, new_total=R * rng.choice([1, 1, 2]), ctx_min=1, ctx_max=_log(rng, 16, 640),
                 prefix=_log(rng, 2, 16384 // c["bt"]) * c["bt"])
    else:
        c.update(window=rng.choice([0, 0, 0, rng.randrange(100, 2000)]), softcap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                 alibi=rng.random() < 0.25, lse=rng.random() < 0.25)
        if rng.random() < 0.55:  # decode, at most 300000 cached tokens in all
            R = _log(rng, 1, 256)
            top = _log(rng, 64, min(131072, 300000 // R))
            c.update(R=R, new_total=R * rng.choice([1, 1, 1, 2, 4]), ctx_min=min(top, rng.randrange(0, 200)),
                     ctx_max=top)
        else:  # prompts and chunks
            R = rng.randrange(1, 7)
            c.update(R=R, new_total=R + _log(rng, 60, 5000), ctx_max=rng.choice([0, _log(rng, 16, 2048)]),
                     docs=rng.choice([0, 0, 3]), bidir=rng.random() < 0.25)
    return c


def _lengths(case):
    """ctx and new of every request: a function of the case alone (its ``mix``)."""
    rng = np.random.default_rng(case["mix"])
    R, total = case["R"], case["new_total"]
    if total % R == 0 and total // R <= 4:
        new = np.full(R, total // R, dtype=np.int64)
    else:
        w = rng.exponential(size=R) ** 2
        new = 1 + np.floor(w / w.sum() * (total - R)).astype(np.int64)
        new[0] += total - new.sum()
    ctx = rng.integers(case["ctx_min"], case["ctx_max"] + 1, size=R)
    ctx[0] = case["ctx_max"]
    return ctx + case["prefix"], new


def _masks(case, ctx, new):
    """doc_start of every new token and bidir_len of every request (None where unused)."""
    rng = np.random.default_rng(case["mix"] + 1)
    doc, bid = None, None
    if case["docs"]:
        parts = []
        for c, n in zip(ctx, new):
            cuts = np.concatenate([[0], np.sort(rng.integers(0, c + n, size=case["docs"] - 1))])
            p = np.arange(c, c + n)
            parts.append(cuts[np.searchsorted(cuts, p, side="right") - 1])
        doc = np.concatenate(parts).astype(np.int32)
    if case["bidir"]:
        bid = rng.integers(0, (ctx + new) // 2 + 1).astype(np.int32)
    return doc, bid


def _bounds(case):
    """Visible keys [lo, hi) of every new token, on the host."""
    ctx, new = _lengths(case)
    doc, bid = _masks(case, ctx, new)
    r = np.repeat(np.arange(case["R"]), new)
    pos = np.arange(new.sum()) - np.repeat(np.cumsum(new) - new, new) + ctx[r]
    lo = np.maximum(0, pos - case["window"] + 1) if case["window"] else np.zeros_like(pos)
    if doc is not None:
        lo = np.maximum(lo, doc)
    hi = pos + 1
    if bid is not None:
        hi = np.minimum(np.maximum(hi, bid[r]), (ctx + new)[r])
    return ctx, new, r, pos, lo, hi


def _cdiv(a, b):
    return -(-a // b)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).to(DEV)


def prepare(case, seed):
    """The paged cache, the step's lengths and new rows; with ``own`` also the attention handle,
    its bound cache and the plan that a program makes once for a step's layers."""
    ctx, new = _lengths(case)
    R, bt, D, N = case["R"], case["bt"], case["D"], int(new.sum())
    dt = DTYPES[case["dtype"]]
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = np.random.default_rng(seed)
    kv = ctx + new
    pages, held = _cdiv(kv, bt), _cdiv(ctx, bt)
    width = int(pages.max())
    common = case["prefix"] // bt
    n_blocks = int((pages - common).sum()) + common + 3
    perm = rng.permutation(n_blocks).astype(np.int32)
    table = np.full((R, width), -1, dtype=np.int32)
    table[:, :common] = perm[:common]
    own_page = (np.arange(width)[None] >= common) & (np.arange(width)[None] < pages[:, None])
    table[own_page] = perm[common:common + int(own_page.sum())]
    st = dict(case=case, R=R, N=N, n_blocks=n_blocks, max_new=int(new.max()), max_kv=int(kv.max()),
              ctx_len=_i32(ctx), new_len=_i32(new))
    if case["op"] == "map":
        fresh = (np.arange(width)[None] >= held[:, None]) & (np.arange(width)[None] < pages[:, None])
        ids = table[fresh].copy()
        table[fresh] = -1
        st["new_ids"] = _i32(ids)
    st["table"] = _i32(table)
    q_start = np.concatenate([[0], np.cumsum(new)])
    r = np.repeat(np.arange(R), new)
    pos = np.arange(N) - q_start[r] + ctx[r]
    if case["op"] == "map":  # written by the call
        st.update(q_start=torch.zeros(R + 1, dtype=torch.int32, device=DEV), kv_len=torch.zeros_like(st["ctx_len"]),
                  slot=torch.zeros(N, dtype=torch.int64, device=DEV), pos=torch.zeros(N, dtype=torch.int32, device=DEV))
    else:
        slot = table[r, pos // bt].astype(np.int64) * bt + pos % bt
        st.update(q_start=_i32(q_start), kv_len=_i32(kv), slot=torch.as_tensor(slot).to(DEV), pos=_i32(pos))
        shape = (n_blocks, bt, case["Hkv"], D)
        st["k_cache"] = torch.randn(shape, dtype=dt, device=DEV, generator=g)
        st["v_cache"] = torch.randn(shape, dtype=dt, device=DEV, generator=g)
    if case["op"] == "append":  # k and v as a fused projection leaves them: slices of one row
        kv_new = torch.randn(N, 2, case["Hkv"], D, dtype=dt, device=DEV, generator=g)
        st["k"], st["v"] = kv_new[:, 0], kv_new[:, 1]
    if case["op"] in ("attn", "shared"):
        st["q"] = torch.randn(N, case["Hq"], D, device=DEV, generator=g).mul_(1.5).to(dt)
        st["o"] = torch.empty(N, case["Hq"], D, dtype=dt, device=DEV)
        st["lse"] = torch.empty(N, case["Hq"], device=DEV) if case["lse"] else None
        st["slopes"] = None
        if case["alibi"]:
            st["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["Hq"] + 1, device=DEV) / case["Hq"])
        doc, bid = _masks(case, ctx, new)
        st["doc_start"] = None if doc is None else _i32(doc)
        st["bidir_len"] = None if bid is None else _i32(bid)
        st["groups"] = _i32([0, R]) if case["prefix"] else None
        st["shared_len"] = _i32([case["prefix"]]) if case["prefix"] else None
    if own:
        _prepare_own(st)
    return st


class _Handle:
    """An attention handle, released with the state that holds it."""

    def __init__(self, pw, desc):
        self.pw, self.h = pw, pw.pw_attn_create(desc)

    def __del__(self):
        self.pw.pw_attn_destroy(self.h)


def _prepare_own(st):
    import any_precision_bit_gb300 as pw
    c = st["case"]
    st["pw"] = pw
    st["handle"] = _Handle(pw, pw.pw_attn_desc(
        L=1, n_heads=c["Hq"], n_kv_heads=c["Hkv"], head_dim=c["D"],
        dtype=pw.PW_BF16 if c["dtype"] == "bf16" else pw.PW_FP16, n_blocks=st["n_blocks"], block_tokens=c["bt"],
        max_requests=c["R"], max_tokens=st["N"], max_shared_tokens=st["N"] if c["prefix"] else 0, n_plans=1, device=0))
    st["step"] = pw.pw_make_step(st["ctx_len"], st["new_len"], st["table"], st["q_start"], st["kv_len"], st["slot"],
                                 st["pos"], max_new=st["max_new"], groups=st.get("groups"),
                                 shared_len=st.get("shared_len"))
    if c["op"] != "map":
        pw.pw_attn_bind(st["handle"].h, 0, st["k_cache"], st["v_cache"])
    if c["op"] in ("attn", "shared"):
        pw.pw_attn_plan(st["handle"].h, 0, st["step"], window=c["window"], doc_start=st["doc_start"],
                        bidir_len=st["bidir_len"], stream=torch.cuda.current_stream())


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "map":
        return _plain_map(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attention(state)


def _own(st, op):
    pw, h, stream = st["pw"], st["handle"].h, torch.cuda.current_stream()
    if op == "map":
        pw.pw_kv_map(h, st["step"], st["new_ids"], stream=stream)
        return {n: st[n] for n in ("table", "q_start", "kv_len", "slot", "pos")}
    if op == "append":
        pw.pw_attn_append(h, 0, st["step"], st["k"], st["v"], stream=stream)
        return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    c = st["case"]
    pw.pw_attn_forward(h, 0, 0, st["q"], st["o"], lse=st["lse"], softcap=c["softcap"], slopes=st["slopes"],
                       stream=stream)
    return {"o": st["o"]} if st["lse"] is None else {"o": st["o"], "lse": st["lse"]}


def _plain_map(st):
    R, N, bt = st["R"], st["N"], st["case"]["bt"]
    ctx, new = st["ctx_len"].long(), st["new_len"].long()
    kv = ctx + new
    held, pages = (ctx + bt - 1) // bt, (kv + bt - 1) // bt
    end, page_end = torch.cumsum(new, 0), torch.cumsum(pages - held, 0)
    table = st["table"].clone()
    i = torch.arange(st["new_ids"].numel(), device=DEV)
    rb = torch.searchsorted(page_end, i, right=True)
    table[rb, held[rb] + i - (page_end - (pages - held))[rb]] = st["new_ids"]
    t = torch.arange(N, device=DEV)
    r = torch.searchsorted(end, t, right=True)
    pos = ctx[r] + t - (end - new)[r]
    slot = table[r, pos // bt].long() * bt + pos % bt
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), end])
    return {"table": table, "q_start": q_start.int(), "kv_len": kv.int(), "slot": slot, "pos": pos.int()}


def _plain_append(st):
    n_blocks, bt, h, d = st["k_cache"].shape
    st["k_cache"].view(n_blocks * bt, h, d)[st["slot"]] = st["k"]
    st["v_cache"].view(n_blocks * bt, h, d)[st["slot"]] = st["v"]
    return {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}


def _plain_attention(st):
    c = st["case"]
    R, Hq, Hkv, D, Tm, Lm = st["R"], c["Hq"], c["Hkv"], c["D"], st["max_new"], st["max_kv"]
    G = Hq // Hkv
    # keys and values of every request, padded: [R, Hkv, L, D]
    blocks = st["table"].long().clamp(min=0)
    k = st["k_cache"][blocks].flatten(1, 2)[:, :Lm].permute(0, 2, 1, 3).float()
    v = st["v_cache"][blocks].flatten(1, 2)[:, :Lm].permute(0, 2, 1, 3).float()
    # queries, padded: [R, Hkv, Tm * G, D]
    start, new = st["q_start"][:-1].long(), st["new_len"].long()
    i = torch.arange(Tm, device=DEV)
    row = (start[:, None] + i[None]).clamp(max=st["N"] - 1)
    q = st["q"][row].float().view(R, Tm, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hkv, Tm * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(R, Hkv, Tm, G, Lm)
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    j = torch.arange(Lm, device=DEV)
    pos = st["ctx_len"].long()[:, None] + i[None]
    if st["slopes"] is not None:
        dist = (pos[:, :, None] - j).abs().float()
        x = x - st["slopes"].view(1, Hkv, 1, G, 1) * dist[:, None, :, None, :]
    lo = torch.zeros_like(pos)
    if c["window"]:
        lo = (pos - c["window"] + 1).clamp(min=0)
    if st["doc_start"] is not None:
        lo = torch.maximum(lo, st["doc_start"].long()[row])
    hi = pos + 1
    if st["bidir_len"] is not None:
        hi = torch.minimum(torch.maximum(hi, st["bidir_len"].long()[:, None]), st["kv_len"].long()[:, None])
    seen = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None, :, None, :]
    x = torch.where(seen, x, torch.full_like(x[:1, :1, :1, :1, :1], -math.inf))
    m = x.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(x - m)
    del x
    s = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(R, Hkv, Tm * G, Lm), v).view(R, Hkv, Tm, G, D) / s
    rr = torch.repeat_interleave(torch.arange(R, device=DEV), new, output_size=st["N"])
    tt = torch.arange(st["N"], device=DEV) - start[rr]
    out = {"o": o.permute(0, 2, 1, 3, 4)[rr, tt].reshape(st["N"], Hq, D).to(st["q"].dtype)}
    if st["lse"] is not None:
        out["lse"] = (m + torch.log(s))[..., 0].permute(0, 2, 1, 3)[rr, tt].reshape(st["N"], Hq)
    return out


def work(case):
    ctx, new, r, pos, lo, hi = _bounds(case)
    R, bt, D, Hq, Hkv, N = case["R"], case["bt"], case["D"], case["Hq"], case["Hkv"], int(new.sum())
    if case["op"] == "map":
        pages = int((_cdiv(ctx + new, bt) - _cdiv(ctx, bt)).sum())
        return {"bytes": 8 * R + 4 * (R + 1) + 4 * R + 8 * pages + 12 * N + 4 * R, "flops": 0}
    if case["op"] == "append":
        return {"bytes": 8 * N + 2 * 2 * 2 * N * Hkv * D, "flops": 0}
    # keys that some new token of the request sees: one span for each request
    first, last = np.full(R, np.iinfo(np.int64).max), np.zeros(R, dtype=np.int64)
    np.minimum.at(first, r, lo)
    np.maximum.at(last, r, hi)
    span = np.maximum(0, last - first)
    keys = int(span.sum()) - case["prefix"] * (R - 1)
    return {"bytes": 2 * keys * Hkv * D * 2 + 2 * N * Hq * D * 2 + 4 * _cdiv(keys, bt) + (4 * N * Hq if case["lse"] else 0),
            "flops": 4 * D * Hq * int((hi - lo).sum())}


def exact(case, seed):
    if case["op"] == "map":  # whole numbers: the plain form's are exact
        return None
    st = prepare(case, seed)
    if case["op"] == "append":
        out = {}
        for name in ("k", "v"):
            cache = st[name + "_cache"].double()
            cache[st["slot"] // case["bt"], st["slot"] % case["bt"]] = st[name].double()
            out[name + "_cache"] = cache
        return out
    ctx, new, r, pos, lo, hi = _bounds(case)
    D, Hq, Hkv, bt = case["D"], case["Hq"], case["Hkv"], case["bt"]
    G, N = Hq // Hkv, st["N"]
    o = torch.zeros(N, Hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(N, Hq, dtype=torch.float64, device=DEV)
    ends = np.cumsum(new)
    head = torch.arange(1, Hq + 1, dtype=torch.float64, device=DEV)
    for i in range(case["R"]):
        b, e, L = int(ends[i] - new[i]), int(ends[i]), int(ctx[i] + new[i])
        blocks = st["table"][i, :_cdiv(L, bt)].long()
        keys = torch.arange(L, device=DEV)
        low, high = (torch.as_tensor(a[b:e]).to(DEV) for a in (lo, hi))
        hide = (keys[None] < low[:, None]) | (keys[None] >= high[:, None])
        if case["alibi"]:
            away = (torch.as_tensor(pos[b:e]).to(DEV)[:, None] - keys[None]).abs().double()
        for h in range(Hkv):
            K = st["k_cache"][blocks][:, :, h].reshape(-1, D)[:L].double()
            V = st["v_cache"][blocks][:, :, h].reshape(-1, D)[:L].double()
            a = torch.einsum("tgd,ld->gtl", st["q"][b:e, h * G:(h + 1) * G].double(), K) / math.sqrt(D)
            if case["softcap"]:
                a = case["softcap"] * torch.tanh(a / case["softcap"])
            if case["alibi"]:
                slope = torch.exp2(-8.0 * head[h * G:(h + 1) * G] / Hq).float().double()
                a = a - slope[:, None, None] * away
            a = a.masked_fill(hide, -math.inf)
            z = torch.logsumexp(a, -1, keepdim=True)
            o[b:e, h * G:(h + 1) * G] = torch.matmul(torch.exp(a - z), V).transpose(0, 1)
            lse[b:e, h * G:(h + 1) * G] = z[..., 0].T
    return {"o": o, "lse": lse} if case["lse"] else {"o": o}
