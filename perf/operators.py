"""Measured cases of the long-context cache operators: windowed attention with sink tokens, attention over a
prefix that a batch shares, the attention weight each cached key collects, and eviction by that weight.

Each case is a dict of plain values.  `run` computes one pass: in the plain form (elementary torch operations in
fp32) where `own` is false, through this package's entry points where it is true.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(name=name, op=op, seqs=1, new_lo=1, new_hi=1, ctx_lo=0, ctx_hi=0, heads=32, kv_heads=8, dim=128,
             block=0, int8=False)
    c.update(kw)
    return c


def listed():
    return [
        # one conversation that streams on under a sliding window: a single decode step, nothing but latency
        _case("sinks decode 1", "sinks", ctx_lo=9001, ctx_hi=9001, window=1024, sinks=4),
        # a serving batch of decode steps over a paged cache, most contexts longer than the window of 4096
        _case("sinks decode 64", "sinks", seqs=64, ctx_lo=1024, ctx_hi=16384, window=4096, sinks=4, block=16),
        # the prefill of one long prompt of a 32-head model under the same window
        _case("sinks prompt 16k", "sinks", new_lo=16384, new_hi=16384, kv_heads=32, window=4096, sinks=4),
        # a few users of one assistant prompt, just started
        _case("prefix decode 8", "prefix", seqs=8, ctx_lo=0, ctx_hi=255, prefix=2047),
        # a batch of decode steps that all ask about the same 32k-token document
        _case("prefix decode 64", "prefix", seqs=64, ctx_lo=256, ctx_hi=4096, prefix=32768),
        # short questions prefilled over a shared prompt held in a paged cache, multi-head attention
        _case("prefix questions 16", "prefix", seqs=16, new_lo=33, new_hi=200, prefix=8191, kv_heads=32, block=16),
        # weight of every cached key for one decode step of a serving batch
        _case("weights decode 64", "weights", seqs=64, ctx_lo=256, ctx_hi=4096),
        # a 512-token chunk over its 4096-token cached prefix, paged cache
        _case("weights chunk 512", "weights", new_lo=512, new_hi=512, ctx_lo=4096, ctx_hi=4096, block=16),
        # the keys of a whole 8k prompt, ranked right after its prefill
        _case("weights prompt 8k", "weights", new_lo=8192, new_hi=8192, kv_heads=32),
        # a few short conversations cut back by a quarter
        _case("evict 4", "evict", seqs=4, ctx_lo=505, ctx_hi=512, budget=384, sinks=4, recent=32),
        # an int8 paged cache of a serving batch, ragged lengths, some already below the budget
        _case("evict int8 64", "evict", seqs=64, ctx_lo=700, ctx_hi=4099, budget=1024, sinks=4, recent=128, block=16,
              int8=True),
        # long prompts squeezed to a quarter after their prefill
        _case("evict 16k", "evict", seqs=16, ctx_lo=16384, ctx_hi=16384, budget=4096, sinks=4, recent=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sinks", "prefix", "weights", "evict"])
    dim = rng.choice([32, 64, 128, 128])
    kv = rng.choice([2, 4, 8, 8, 16, 32])
    group = rng.choice([1, 2, 4, 4, 8])
    while kv * group > 64:
        group //= 2
    c = _case("", op, dim=dim, kv_heads=kv, heads=kv * group, block=rng.choice([0, 0, 16, 64]),
              int8=rng.random() < 0.25)
    del c["name"]
    seqs = _log(rng, 1, 64)
    ctx = _log(rng, 17, 16384)
    while seqs * ctx * kv * dim > 1 << 29:  # the cache: at most 1 GiB of bf16 keys
        seqs, ctx = max(1, seqs * 2 // 3), max(17, ctx * 3 // 4)
    new = 1
    if op != "evict" and rng.random() < 0.4:  # a prefill or a chunk
        new = _log(rng, 2, 4096)
        while seqs * new * (new + ctx) * kv * group > 1 << 31:
            seqs, new = max(1, seqs // 2), max(2, new * 3 // 4)
    c.update(seqs=seqs, ctx_lo=max(0, ctx // rng.choice([1, 2, 8])), ctx_hi=ctx, new_hi=new,
             new_lo=max(1, new // rng.choice([1, 3])))
    if op == "sinks":
        c.update(window=_log(rng, 64, 4096), sinks=_log(rng, 1, 256))
    if op == "prefix":
        pre = _log(rng, 64, 32768)
        while seqs * new * pre * kv * group > 1 << 31 or pre * kv * dim > 1 << 28:
            pre = max(64, pre // 2)
        c.update(prefix=pre)
    if op == "evict":
        budget = max(1, int(ctx * rng.uniform(0.2, 0.95)))
        sinks = min(budget // 4, 4)
        c.update(budget=budget, sinks=sinks, recent=min(budget - sinks, budget // rng.choice([4, 8])))
    return c


def _spread(n, lo, hi):
    """n lengths spread over [lo, hi] (golden-ratio steps: the same for every seed, in no order)."""
    return [lo + int((hi - lo + 1) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(n)]


def _lengths(c):
    """(new tokens, cached tokens) of each sequence."""
    return _spread(c["seqs"], c["new_lo"], c["new_hi"]), _spread(c["seqs"], c["ctx_lo"], c["ctx_hi"])[::-1]


def _visible(n, p, window, sinks):
    """(query, key) pairs that a causal sequence of n new tokens over p cached ones sees."""
    if not window:
        return n * p + n * (n + 1) // 2
    tot = 0
    for i in range(n):
        tot += min(p + i + 1, window) + max(0, min(sinks, p + i + 1 - window))
    return tot


def work(case):
    c = case
    d, H, Hk = c["dim"], c["heads"], c["kv_heads"]
    new, ctx = _lengths(c)
    T = sum(new)
    row = d + 4 if c["int8"] else 2 * d  # bytes of one cached key or value row
    if c["op"] == "evict":
        moved = sum(c["budget"] for p in ctx if p > c["budget"]) * Hk
        kept = sum(min(p, c["budget"]) for p in ctx) * Hk
        return {"bytes": 2 * 2 * row * moved + 4 * sum(ctx) * Hk + (4 + 4) * kept, "flops": 0}
    window, sinks, pre = c.get("window", 0), c.get("sinks", 0), c.get("prefix", 0)
    pairs = sum(_visible(n, p, window, sinks) for n, p in zip(new, ctx)) + T * pre
    if window:  # the cached keys that some new token sees
        read = sum(p if p < window + sinks else window - 1 + sinks for p in ctx)
    else:
        read = sum(ctx)
    read += pre
    if c["op"] == "weights":
        w = 4 * Hk * (2 * sum(ctx) + T)
        return {"bytes": 2 * T * (H + Hk) * d + 4 * T * H + read * Hk * row + w, "flops": 2 * d * H * pairs}
    return {"bytes": 2 * T * (2 * H + 2 * Hk) * d + 4 * T * H + 2 * read * Hk * row + 2 * T * Hk * row,
            "flops": 4 * d * H * pairs}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if math.prod(shape) < 1 << 24
                       else torch.bfloat16).to(torch.bfloat16)


def _cache(g, c, shape):
    """(keys or values, row scales or None) of a cache of [..., rows, dim]."""
    if not c["int8"]:
        return _randn(g, *shape), None
    codes = torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)
    return codes, torch.rand(shape[:-1], generator=g, device=DEV) * 0.012 + 0.008


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    new, ctx = _lengths(c)
    B, T, d, H, Hk, bs = c["seqs"], sum(new), c["dim"], c["heads"], c["kv_heads"], c["block"]
    evict = c["op"] == "evict"
    cap = max(p if evict else n + p for n, p in zip(new, ctx))
    pre = c.get("prefix", 0)
    s = dict(case=c, B=B, T=T, scale=1.0 / math.sqrt(d), table=None, prefix_table=None)
    i32 = dict(dtype=torch.int32, device=DEV)
    if bs:
        blocks = -(-cap // bs)
        cap = blocks * bs
        pre_blocks = -(-pre // bs)
        order = torch.randperm(B * blocks + pre_blocks + 3, generator=g, device=DEV).to(torch.int32)
        s["table"] = order[:B * blocks].reshape(B, blocks).contiguous()
        s["prefix_table"] = order[B * blocks:B * blocks + pre_blocks].contiguous()
        shape = (B * blocks + pre_blocks + 3, Hk, bs, d)
    else:
        shape = (B, Hk, cap, d)
    s["cap"] = cap
    s["ck"], s["sk"] = _cache(g, c, shape)
    s["cv"], s["sv"] = _cache(g, c, shape)
    s["offsets"] = torch.tensor(ctx, **i32)
    if evict:
        # weights as attention leaves them: mostly small, a few keys with much of it, and ties at zero
        w = torch.rand(shape[:-1], generator=g, device=DEV)
        s["weights"] = torch.where(w < 0.05, 0.0, w ** 6 * 40)
        s["kept_weights"] = torch.zeros_like(s["weights"])
        s["kept_lengths"] = torch.zeros_like(s["offsets"])
        s["kept_index"] = torch.zeros((B, Hk, c["budget"]), **i32)
        return s
    if pre and not bs:
        s["pk"], s["psk"] = _cache(g, c, (Hk, pre, d))
        s["pv"], s["psv"] = _cache(g, c, (Hk, pre, d))
    s["q"], s["k"], s["v"] = _randn(g, T, H, d), _randn(g, T, Hk, d), _randn(g, T, Hk, d)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ck = [0]
    for n, p in zip(new, ctx):
        ck.append(ck[-1] + n + p)
    s["cu_q"], s["cu_k"] = torch.tensor(cu, **i32), torch.tensor(ck, **i32)
    s["out"] = torch.zeros((T, H, d), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((T, H), dtype=torch.float32, device=DEV)
    if c["op"] == "weights":
        s["lse"] = _plain_scores(s, _padded(s))[1]  # what the attention call of this step left
        s["weights"] = torch.rand(shape[:-1], generator=g, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------

def _rows(s, name, rows):
    """Index of the first `rows` cache rows of each sequence in s[name], as [B, Hk, rows] of it."""
    x = s[name]
    if s["table"] is None:
        return x[:, :, :rows]
    bs = s["case"]["block"]
    y = x[s["table"][:, :-(-rows // bs)].long()]                # [B, blocks, Hk, bs, ...]
    y = y.transpose(1, 2).reshape(s["B"], x.shape[1], -1, *x.shape[3:])
    return y[:, :, :rows]


def _f32(s, name, scale, rows):
    x = _rows(s, name, rows).float()
    return x * _rows(s, scale, rows)[..., None] if s[scale] is not None else x


def _prefix(s, which):
    """The shared prefix's keys ("k") or values ("v"): [Hk, prefix, dim]."""
    c = s["case"]
    if s["table"] is None:
        x, sc = s["p" + which], s["ps" + which]
    else:
        at = s["prefix_table"].long()
        x = s["c" + which][at].transpose(0, 1).reshape(c["kv_heads"], -1, c["dim"])[:, :c["prefix"]]
        sc = s["s" + which]
        if sc is not None:
            sc = sc[at].transpose(0, 1).reshape(c["kv_heads"], -1)[:, :c["prefix"]]
    return x.float() if sc is None else x.float() * sc[..., None]


def _padded(s):
    """Where the tokens sit in a batch padded to its longest sequence."""
    cu, off = s["cu_q"].long(), s["offsets"].long()
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    c = s["case"]
    new, ctx = _lengths(c)
    n, rows = max(new), max(x + y for x, y in zip(new, ctx))
    return dict(b=b, i=i, pos=off[b] + i, n=n, rows=rows)


def _plain_scores(s, at):
    """exp(score - row maximum) of every query against its sequence's keys, [B, Hk, G, n, rows], the shared
    prefix's part [Hk, T, G, prefix] or None, the lse of every row, and the row maxima and sums."""
    c = s["case"]
    B, Hk, G, d, n = s["B"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"], at["n"]
    k = _f32(s, "ck", "sk", at["rows"]).clone()
    k[at["b"], :, at["pos"]] = s["k"].float()
    q = torch.zeros((B, n, Hk, G, d), device=DEV)
    q[at["b"], at["i"]] = s["q"].float().reshape(-1, Hk, G, d)
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, d), k.transpose(2, 3)).reshape(B, Hk, G, n, -1)
    x.mul_(s["scale"])
    j = torch.arange(at["rows"], device=DEV)
    p = s["offsets"].long()[:, None] + torch.arange(n, device=DEV)      # absolute position of each query
    hide = j > p[..., None]
    if c.get("window"):
        hide |= (j <= p[..., None] - c["window"]) & (j >= c["sinks"])
    x.masked_fill_(hide[:, None, None], -math.inf)
    m = x.amax(-1)                                                     # [B, Hk, G, n]
    y = None
    if c.get("prefix"):
        qt = s["q"].float().reshape(-1, Hk, G, d).permute(1, 0, 2, 3).reshape(Hk, -1, d)
        y = torch.matmul(qt, _prefix(s, "k").transpose(1, 2)).mul_(s["scale"]).reshape(Hk, s["T"], G, -1)
        my = torch.full((B, n, Hk, G), -math.inf, device=DEV)
        my[at["b"], at["i"]] = y.amax(-1).permute(1, 0, 2)
        m = torch.maximum(m, my.permute(0, 2, 3, 1))
    x.sub_(m[..., None]).exp_()
    z = x.sum(-1)
    mt = m.permute(0, 3, 1, 2)[at["b"], at["i"]]                        # [T, Hk, G]
    zt = z.permute(0, 3, 1, 2)[at["b"], at["i"]]
    if y is not None:
        y.sub_(mt.permute(1, 0, 2)[..., None]).exp_()
        zt = zt + y.sum(-1).permute(1, 0, 2)
    lse = (mt + zt.log()).reshape(s["T"], -1)
    return x, lse, y, zt


def _store(s, at, which):
    """The new tokens' rows into the cache."""
    x = s[which]
    rows = (at["b"], slice(None), at["pos"])
    if s["table"] is not None:
        bs = s["case"]["block"]
        rows = (s["table"].long()[at["b"], at["pos"] // bs], slice(None), at["pos"] % bs)
    if s["s" + which] is not None:
        x = x.float()
        sc = x.abs().amax(-1) / 127.0
        x = torch.where(sc[..., None] > 0, (x / sc[..., None]).round().clamp(-127, 127), 0.0).to(torch.int8)
        s["s" + which][rows] = sc
    s["c" + which][rows] = x


def _plain_attention(s):
    c, at = s["case"], _padded(s)
    B, Hk, G, n = s["B"], c["kv_heads"], c["heads"] // c["kv_heads"], at["n"]
    x, lse, y, z = _plain_scores(s, at)
    v = _f32(s, "cv", "sv", at["rows"]).clone()
    v[at["b"], :, at["pos"]] = s["v"].float()
    o = torch.matmul(x.reshape(B, Hk, G * n, -1), v).reshape(B, Hk, G, n, -1)
    o = o.permute(0, 3, 1, 2, 4)[at["b"], at["i"]]                      # [T, Hk, G, d]
    if y is not None:
        o = o + torch.matmul(y.reshape(Hk, s["T"] * G, -1), _prefix(s, "v")).reshape(Hk, s["T"], G, -1).transpose(0, 1)
    s["out"].copy_((o / z[..., None]).reshape(s["out"].shape))
    s["lse"].copy_(lse)
    _store(s, at, "k")
    _store(s, at, "v")


def _plain_weights(s):
    c, at = s["case"], _padded(s)
    B, Hk, G, n = s["B"], c["kv_heads"], c["heads"] // c["kv_heads"], at["n"]
    k = _f32(s, "ck", "sk", at["rows"]).clone()
    k[at["b"], :, at["pos"]] = s["k"].float()
    q = torch.zeros((B, n, Hk, G, c["dim"]), device=DEV)
    q[at["b"], at["i"]] = s["q"].float().reshape(-1, Hk, G, c["dim"])
    lse = torch.full((B, n, Hk, G), math.inf, device=DEV)
    lse[at["b"], at["i"]] = s["lse"].reshape(-1, Hk, G)
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, -1), k.transpose(2, 3)).reshape(B, Hk, G, n, -1)
    x.mul_(s["scale"]).sub_(lse.permute(0, 2, 3, 1)[..., None]).exp_()
    p = s["offsets"].long()[:, None] + torch.arange(n, device=DEV)
    j = torch.arange(at["rows"], device=DEV)
    x.masked_fill_((j > p[..., None])[:, None, None], 0.0)
    add = x.sum((2, 3))                                                # [B, Hk, rows]
    off, end = s["offsets"].long()[:, None, None], (s["cu_k"][1:] - s["cu_k"][:-1]).long()[:, None, None]
    old = _rows(s, "weights", at["rows"])
    got = torch.where(j < off, old + add, torch.where(j < end, add, old))
    if s["table"] is None:
        s["weights"][:, :, :at["rows"]] = got
    else:
        bs = c["block"]
        t = s["table"].long()[:, j // bs]                              # [B, rows]
        s["weights"][t, :, j % bs] = got.transpose(1, 2)


def _plain_evict(s):
    c = s["case"]
    budget, sinks, recent = c["budget"], c["sinks"], c["recent"]
    rows = max(_lengths(c)[1])
    ln = s["offsets"].long()[:, None, None]
    w = _rows(s, "weights", rows)
    j = torch.arange(rows, device=DEV)
    # rank: forced tokens first, then by weight (ties: lowest position first), tokens past the end last
    forced = (j < sinks) | (j >= ln - recent)
    key = torch.where((j < ln) & ~forced, w, torch.where(j < ln, math.inf, -math.inf))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    kept = order[..., :budget]
    count = torch.minimum(ln, torch.tensor(budget, device=DEV))        # [B, 1, 1]
    slot = torch.arange(kept.shape[-1], device=DEV)
    kept = torch.where(slot < count, kept, rows).sort(-1).values       # ascending positions
    here = (slot < count).expand(kept.shape)
    s["kept_index"].fill_(-1)
    s["kept_index"][..., :kept.shape[-1]] = torch.where(here, kept, -1)
    s["kept_lengths"].copy_(count.reshape(-1))
    src = torch.where(here, kept, slot)
    B, Hk = kept.shape[:2]
    b = torch.arange(B, device=DEV)[:, None, None].expand(kept.shape)
    h = torch.arange(Hk, device=DEV)[None, :, None].expand(kept.shape)
    b, h, src, dst = b[here], h[here], src[here], slot.expand(kept.shape)[here]
    if s["table"] is None:
        at_src, at_dst = (b, h, src), (b, h, dst)
    else:
        bs, t = c["block"], s["table"].long()
        at_src, at_dst = (t[b, src // bs], h, src % bs), (t[b, dst // bs], h, dst % bs)
    s["kept_weights"][at_dst] = s["weights"][at_src]
    for name in ("ck", "cv", "sk", "sv"):
        if s[name] is not None:
            s[name][at_dst] = s[name][at_src]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _values(s, which):
    """The whole cache as the values that it holds."""
    x = s["c" + which]
    return x if s["s" + which] is None else x.float() * s["s" + which][..., None]


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        {"sinks": _plain_attention, "prefix": _plain_attention, "weights": _plain_weights, "evict": _plain_evict}[op](s)
    else:
        from prefill_phase_attention_gb300 import binding as B
        cache = dict(block_table=s["table"], cache_k_scale=s["sk"], cache_v_scale=s["sv"])
        if op == "sinks":
            B.prefill_attn_varlen_sinks(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["ck"], s["cv"], s["offsets"],
                                        s["out"], s["lse"], window=c["window"], sink_tokens=c["sinks"],
                                        scale=s["scale"], **cache)
        elif op == "prefix":
            pre = dict(prefix_table=s["prefix_table"], prefix_len=c["prefix"]) if s["table"] is not None else \
                dict(prefix_k=s["pk"], prefix_v=s["pv"], prefix_k_scale=s["psk"], prefix_v_scale=s["psv"])
            B.prefill_attn_varlen_prefix(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["ck"], s["cv"], s["offsets"],
                                         s["out"], s["lse"], scale=s["scale"], **pre, **cache)
        elif op == "weights":
            B.prefill_attn_key_weights(s["q"], s["k"], s["cu_q"], s["cu_k"], s["ck"], s["offsets"], s["lse"],
                                       s["weights"], scale=s["scale"], block_table=s["table"], cache_k_scale=s["sk"])
        else:
            B.prefill_attn_evict(s["ck"], s["cv"], s["weights"], s["offsets"], s["kept_lengths"], s["kept_index"],
                                 s["kept_weights"], budget=c["budget"], sink_tokens=c["sinks"],
                                 recent_tokens=c["recent"], **cache)
    if op == "weights":
        return {"weights": s["weights"]}
    got = {"cache_k": s["ck"], "cache_v": s["cv"]}
    if c["int8"]:
        got = {"cache_k": _values(s, "k"), "cache_v": _values(s, "v")}
    if op == "evict":
        return {**got, "weights": s["kept_weights"], "lengths": s["kept_lengths"], "index": s["kept_index"]}
    return {"out": s["out"], "lse": s["lse"], **got}


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence and one KV head at a time
# ---------------------------------------------------------------------------

def _where(s, b, rows):
    """(slot, row) of the first `rows` positions of sequence b in the cache tensors."""
    if s["table"] is None:
        return torch.full((rows,), b, device=DEV), torch.arange(rows, device=DEV)
    bs = s["case"]["block"]
    pos = torch.arange(rows, device=DEV)
    return s["table"][b, pos // bs].long(), pos % bs


def _take64(s, which, b, h, rows):
    slot, row = _where(s, b, rows)
    x = s["c" + which][slot, h, row] if s["table"] is not None else s["c" + which][b, h, :rows]
    x = x.double()
    if s["s" + which] is not None:
        sc = s["s" + which][slot, h, row] if s["table"] is not None else s["s" + which][b, h, :rows]
        x = x * sc.double()[:, None]
    return x


def _prefix64(s, which, h):
    c = s["case"]
    if s["table"] is None:
        x = s["p" + which][h].double()
        return x if s["ps" + which] is None else x * s["ps" + which][h].double()[:, None]
    bs = c["block"]
    pos = torch.arange(c["prefix"], device=DEV)
    blk = s["prefix_table"][pos // bs].long()
    x = s["c" + which][blk, h, pos % bs].double()
    return x if s["s" + which] is None else x * s["s" + which][blk, h, pos % bs].double()[:, None]


def _exact_pairs(c):
    new, ctx = _lengths(c)
    span = lambda n, p: n * min(p + n, c["window"] + c["sinks"] + 512 if c.get("window") else p + n)  # noqa: E731
    return c["heads"] * sum(span(n, p) + n * c.get("prefix", 0) for n, p in zip(new, ctx))


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    new, ctx = _lengths(c)
    H, Hk = c["heads"], c["kv_heads"]
    G = H // Hk
    if c["op"] == "evict":
        return _exact_evict(s, new, ctx)
    if _exact_pairs(c) * c["dim"] > 1 << 41:
        return None
    window, sinks, scale = c.get("window", 0), c.get("sinks", 0), s["scale"]
    out = torch.zeros((s["T"], H, c["dim"]), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["T"], H), dtype=torch.float64, device=DEV)
    weights = s["weights"].double() if c["op"] == "weights" else None
    for h in range(Hk):
        pk = _prefix64(s, "k", h) if c.get("prefix") else None
        pv = _prefix64(s, "v", h) if c.get("prefix") else None
        t0 = 0
        for b, (n, p) in enumerate(zip(new, ctx)):
            k = torch.cat([_take64(s, "k", b, h, p), s["k"][t0:t0 + n, h].double()])
            v = torch.cat([_take64(s, "v", b, h, p), s["v"][t0:t0 + n, h].double()])
            add = torch.zeros(p + n, dtype=torch.float64, device=DEV)
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                first = max(0, p + i0 - window + 1) if window else 0
                j = torch.arange(first, p + i1, device=DEV)
                if first > 0:
                    j = torch.cat([torch.arange(min(sinks, first), device=DEV), j])
                at = torch.arange(p + i0, p + i1, device=DEV)[:, None]
                see = j <= at
                if window:
                    see &= (at - j < window) | (j < sinks)
                q = s["q"][t0 + i0:t0 + i1, h * G:(h + 1) * G].double()          # [i, G, d]
                x = torch.einsum("igd,jd->igj", q, k[j]) * scale
                x = torch.where(see[:, None], x, -math.inf)
                if weights is not None:
                    e = torch.exp(x - s["lse"][t0 + i0:t0 + i1, h * G:(h + 1) * G].double()[..., None])
                    add[j] += e.sum((0, 1))
                    continue
                val = v[j]
                if pk is not None:
                    x = torch.cat([x, torch.einsum("igd,jd->igj", q, pk) * scale], -1)
                    val = torch.cat([val, pv])
                z = torch.logsumexp(x, -1)
                out[t0 + i0:t0 + i1, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", torch.exp(x - z[..., None]), val)
                lse[t0 + i0:t0 + i1, h * G:(h + 1) * G] = z
            if weights is not None:
                slot, row = _where(s, b, p + n)
                if s["table"] is None:
                    weights[b, h, :p] += add[:p]
                    weights[b, h, p:p + n] = add[p:]
                else:
                    weights[slot[:p], h, row[:p]] += add[:p]
                    weights[slot[p:], h, row[p:]] = add[p:]
            t0 += n
    if weights is not None:
        return {"weights": weights}
    caches = {}
    for which in ("k", "v"):
        x = s["c" + which]
        if c["int8"]:
            caches["cache_" + which] = None
            continue
        t0 = 0
        for b, (n, p) in enumerate(zip(new, ctx)):
            slot, row = _where(s, b, p + n)
            if s["table"] is None:
                x[b, :, p:p + n] = s[which][t0:t0 + n].transpose(0, 1)
            else:
                x[slot[p:], :, row[p:]] = s[which][t0:t0 + n]
            t0 += n
        caches["cache_" + which] = x
    return {"out": out, "lse": lse, **caches}


def _exact_evict(s, new, ctx):
    c = s["case"]
    budget, sinks, recent = c["budget"], c["sinks"], c["recent"]
    whole = {n: s[n].clone() for n in ("ck", "cv", "sk", "sv") if s[n] is not None}
    kept_w, index = s["kept_weights"].clone(), torch.full_like(s["kept_index"], -1)
    for b, p in enumerate(ctx):
        m = min(p, budget)
        slot, row = _where(s, b, p)
        for h in range(c["kv_heads"]):
            pick = (lambda x: x[b, h, :p]) if s["table"] is None else (lambda x: x[slot, h, row])  # noqa: E731
            w = pick(s["weights"])
            if p <= budget:
                keep = torch.arange(p, device=DEV)
            else:
                mid = w[sinks:p - recent]
                best = torch.sort(mid, dim=-1, descending=True, stable=True).indices[:budget - sinks - recent] + sinks
                keep = torch.cat([torch.arange(sinks, device=DEV), best.sort().values,
                                  torch.arange(p - recent, p, device=DEV)])
            index[b, h, :m] = keep.to(torch.int32)
            for x, y in [(kept_w, s["weights"])] + [(whole[n], s[n]) for n in whole]:
                if s["table"] is None:
                    x[b, h, :m] = y[b, h, keep]
                else:
                    x[slot[:m], h, row[:m]] = y[slot[keep], h, row[keep]]
    got = {"cache_" + w: whole["c" + w] if s["s" + w] is None else whole["c" + w].float() * whole["s" + w][..., None]
           for w in ("k", "v")}
    return {**got, "weights": kept_w, "lengths": torch.tensor([min(p, budget) for p in ctx], dtype=torch.int32,
                                                              device=DEV), "index": index}
