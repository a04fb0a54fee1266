"""Measured cases of the 4-bit KV cache: attention over it (which also writes the new tokens), quantising keys and
values into it, and reading it back.

A row (token, KV head) is cut into groups of channels; a group holds the scale s and the minimum m (bf16) and a
4-bit code c per channel, and stands for m + c s.

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
             group=128, block=0, window=0)
    c.update(kw)
    return c


def listed():
    return [
        # one conversation's decode step: nothing but latency
        _case("attend decode 1", "attend", ctx_lo=9001, ctx_hi=9001),
        # a serving batch of decode steps over a paged cache
        _case("attend decode 64", "attend", seqs=64, ctx_lo=256, ctx_hi=4096, block=16),
        # the same with long contexts and small groups (the more exact format)
        _case("attend decode long", "attend", seqs=64, ctx_lo=1024, ctx_hi=16384, group=32),
        # drafts of 5 tokens verified at once, heads of 64
        _case("attend draft 16", "attend", seqs=16, new_lo=5, new_hi=5, ctx_lo=500, ctx_hi=8000, dim=64, group=64),
        # a 512-token chunk of a prompt over its 4096 cached tokens, beside nothing else
        _case("attend chunk 512", "attend", new_lo=512, new_hi=512, ctx_lo=4096, ctx_hi=4096, block=16, group=64),
        # a long second turn: 4096 new tokens over 4096 cached ones, multi-head attention
        _case("attend turn 4k", "attend", new_lo=4096, new_hi=4096, ctx_lo=4096, ctx_hi=4096, kv_heads=32),
        # (the write cases read what they wrote back, as a check or a bf16 consumer does)
        # the keys and values of one decode step, computed elsewhere, into pages
        _case("write step 64", "write", seqs=64, ctx_lo=256, ctx_hi=4096, block=16),
        # prompts of many lengths, small groups
        _case("write prompts 16", "write", seqs=16, new_lo=10, new_hi=2048, kv_heads=32, group=32),
        # a bf16 prompt of 32768 tokens squeezed into 4 bits
        _case("write prompt 32k", "write", new_lo=32768, new_hi=32768, kv_heads=32),
        # a few short conversations back to bf16
        _case("read 4", "read", seqs=4, new_lo=505, new_hi=512),
        # a batch out of pages, heads of 64 with small groups
        _case("read pages 64", "read", seqs=64, new_lo=700, new_hi=4099, dim=64, group=32, block=16),
        # long caches back to bf16, behind what stays in 4 bits
        _case("read 16k", "read", seqs=16, new_lo=16384, new_hi=16384, ctx_lo=0, ctx_hi=100, group=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read"])
    dim = rng.choice([32, 64, 128, 128])
    kv = rng.choice([1, 2, 4, 8, 8, 16, 32])
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    share = rng.choice([1, 2, 4, 4, 8, 16])
    while kv * share > 64:
        share //= 2
    c = _case("", op, dim=dim, kv_heads=kv, heads=kv * share, group=group, block=rng.choice([0, 0, 8, 16, 64]))
    del c["name"]
    seqs = _log(rng, 1, 64)
    ctx = _log(rng, 17, 16384)
    while seqs * ctx * kv * dim > 1 << 29:
        seqs, ctx = max(1, seqs * 2 // 3), max(17, ctx * 3 // 4)
    new = 1
    if op == "attend":
        if rng.random() < 0.5:  # a chunk, a draft or a prompt
            new = _log(rng, 2, 4096)
            while seqs * new * (new + ctx) * kv * share > 1 << 30:
                seqs, new = max(1, seqs // 2), max(2, new * 3 // 4)
        if rng.random() < 0.2:
            c["window"] = _log(rng, 16, 4096)
    else:
        new, ctx = ctx, _log(rng, 1, 1000) * rng.choice([0, 1])
    c.update(seqs=seqs, ctx_lo=ctx // rng.choice([1, 2, 8]), ctx_hi=ctx, new_hi=new,
             new_lo=max(1, new // rng.choice([1, 3])))
    return c


def _spread(n, lo, hi):
    """n lengths spread over [lo, hi] (golden-ratio steps: the same for every seed, in no order)."""
    return [lo + int((hi - lo + 1) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(n)]


def _lengths(c):
    """(tokens of the call, cached tokens ahead of them) of each sequence."""
    return _spread(c["seqs"], c["new_lo"], c["new_hi"]), _spread(c["seqs"], c["ctx_lo"], c["ctx_hi"])[::-1]


def _visible(n, p, window):
    """(query, key) pairs that a causal sequence of n new tokens over p cached ones sees."""
    if not window:
        return n * p + n * (n + 1) // 2
    return sum(min(p + i + 1, window) for i in range(n))


def work(case):
    c = case
    d, H, Hk = c["dim"], c["heads"], c["kv_heads"]
    new, ctx = _lengths(c)
    T = sum(new)
    row = d // 2 + 4 * (d // c["group"])     # bytes of one row of the cache
    if c["op"] != "attend":
        once = 2 * T * Hk * (2 * d + row)     # k and v one way and the cache's rows the other
        return {"bytes": 2 * once if c["op"] == "write" else once, "flops": 0}
    pairs = sum(_visible(n, p, c["window"]) for n, p in zip(new, ctx))
    read = sum(min(p, c["window"] - 1) if c["window"] else p for p in ctx)
    # q, out, lse; the new k and v; the cached rows; the new rows written, then read back as bf16
    return {"bytes": 2 * 2 * T * H * d + 4 * T * H + 2 * 2 * T * Hk * d + 2 * read * Hk * row
            + 2 * T * Hk * (2 * row + 2 * d), "flops": 4 * d * H * pairs}


# ---------------------------------------------------------------------------
# the format
# ---------------------------------------------------------------------------

def _quantise(x, group):
    """(codes uint8 [..., d / 2], params bf16 [..., d / group, 2]) of bf16 rows x [..., d]."""
    x = x.float().unflatten(-1, (-1, group))
    lo, hi = x.amin(-1), x.amax(-1)
    s = ((hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32, device=x.device)).to(torch.bfloat16)
    s = torch.where(s.float() >= 2.0 ** -126, s, 0.0)
    r = torch.where(s > 0, torch.reciprocal(s.float()), 0.0)
    code = torch.round((x - lo[..., None]) * r[..., None]).clamp(max=15).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.stack([s, lo.to(torch.bfloat16)], -1)


def _values(codes, params):
    """fp32 values of rows (codes [..., d / 2], params [..., d / group, 2])."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    p = params.float()
    return (c.unflatten(-1, (p.shape[-2], -1)) * p[..., 0:1] + p[..., 1:2]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32 if math.prod(shape) < 1 << 24
                       else torch.bfloat16).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    new, ctx = _lengths(c)
    B, T, d, H, Hk, bs = c["seqs"], sum(new), c["dim"], c["heads"], c["kv_heads"], c["block"]
    cap = max(n + p for n, p in zip(new, ctx))
    s = dict(case=c, B=B, T=T, scale=1.0 / math.sqrt(d), table=None)
    i32 = dict(dtype=torch.int32, device=DEV)
    slots, rows = B, cap
    if bs:
        blocks = -(-cap // bs)
        order = torch.randperm(B * blocks + 3, generator=g, device=DEV).to(torch.int32)
        s["table"] = order[:B * blocks].reshape(B, blocks).contiguous()
        slots, rows = B * blocks + 3, bs
    # keys as models have them: some channels far from zero in every token
    offset = torch.randn((Hk, 1, d), generator=g, device=DEV) ** 3
    for which in ("k", "v"):
        codes = torch.empty((slots, Hk, rows, d // 2), dtype=torch.uint8, device=DEV)
        params = torch.empty((slots, Hk, rows, d // c["group"], 2), dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 25) // (Hk * rows * d))
        for i in range(0, slots, step):
            x = torch.randn((min(step, slots - i), Hk, rows, d), generator=g, device=DEV)
            if which == "k":
                x += offset
            codes[i:i + step], params[i:i + step] = _quantise(x.to(torch.bfloat16), c["group"])
        s["c" + which], s["p" + which] = codes, params
        x = _randn(g, T, Hk, d)
        s[which] = (x + offset.to(torch.bfloat16)[:, 0]) if which == "k" else x
    cu, ck = [0], [0]
    for n, p in zip(new, ctx):
        cu.append(cu[-1] + n)
        ck.append(ck[-1] + n + p)
    s["cu_q"], s["cu_k"] = torch.tensor(cu, **i32), torch.tensor(ck, **i32)
    s["offsets"] = torch.tensor(ctx, **i32)
    s["k_back"], s["v_back"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    if c["op"] == "attend":
        s["q"] = _randn(g, T, H, d)
        s["out"] = torch.zeros((T, H, d), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.zeros((T, H), dtype=torch.float32, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------

def _places(s):
    """Where the call's tokens are: sequence, index in it, position, and (slot, row) in the cache tensors."""
    cu, off = s["cu_q"].long(), s["offsets"].long()
    t = torch.arange(s["T"], device=DEV)
    b = torch.searchsorted(cu, t, right=True) - 1
    i = t - cu[b]
    pos = off[b] + i
    if s["table"] is None:
        return b, i, pos, b, pos
    bs = s["case"]["block"]
    return b, i, pos, s["table"].long()[b, pos // bs], pos % bs


def _plain_write(s):
    _, _, _, slot, row = _places(s)
    for which in ("k", "v"):
        codes, params = _quantise(s[which], s["case"]["group"])
        s["c" + which][slot, :, row] = codes
        s["p" + which][slot, :, row] = params


def _plain_read(s):
    _, _, _, slot, row = _places(s)
    for which in ("k", "v"):
        s[which + "_back"].copy_(_values(s["c" + which][slot, :, row], s["p" + which][slot, :, row]))


def _cached(s, which, rows):
    """Values of the first `rows` cache rows of each sequence, [B, Hk, rows, d]."""
    codes, params = s["c" + which], s["p" + which]
    if s["table"] is not None:
        bs = s["case"]["block"]
        at = s["table"][:, :-(-rows // bs)].long()
        codes, params = codes[at].transpose(1, 2).flatten(2, 3), params[at].transpose(1, 2).flatten(2, 3)
    return _values(codes[:, :, :rows], params[:, :, :rows])


def _plain_attend(s):
    c = s["case"]
    new, ctx = _lengths(c)
    n, rows = max(new), max(x + y for x, y in zip(new, ctx))
    B, Hk, G, d = s["B"], c["kv_heads"], c["heads"] // c["kv_heads"], c["dim"]
    b, i, pos, _, _ = _places(s)
    k, v = _cached(s, "k", rows), _cached(s, "v", rows)
    k[b, :, pos], v[b, :, pos] = s["k"].float(), s["v"].float()      # the new tokens at full precision
    j = torch.arange(rows, device=DEV)
    v.masked_fill_((j >= s["offsets"][:, None] + (s["cu_q"][1:] - s["cu_q"][:-1])[:, None])[:, None, :, None], 0.0)
    q = torch.zeros((B, n, Hk, G, d), device=DEV)
    q[b, i] = s["q"].float().reshape(-1, Hk, G, d)
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, Hk, G * n, d), k.transpose(2, 3)).reshape(B, Hk, G, n, -1)
    x.mul_(s["scale"])
    p = s["offsets"].long()[:, None] + torch.arange(n, device=DEV)
    hide = j > p[..., None]
    if c["window"]:
        hide |= j <= p[..., None] - c["window"]
    x.masked_fill_(hide[:, None, None], -math.inf)
    m = x.amax(-1)
    m = torch.where(m == -math.inf, 0.0, m)                           # rows of the padding may see no key
    x.sub_(m[..., None]).exp_()
    z = x.sum(-1)
    o = torch.matmul(x.reshape(B, Hk, G * n, -1), v).reshape(B, Hk, G, n, -1) / z[..., None]
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[b, i].reshape(s["out"].shape))
    s["lse"].copy_((m + z.log()).permute(0, 3, 1, 2)[b, i].reshape(s["lse"].shape))
    _plain_write(s)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        if op == "attend":
            _plain_attend(s)
        elif op == "write":
            _plain_write(s)
        _plain_read(s)
    else:
        from prefill_phase_attention_gb300 import binding as B
        cache = dict(cache_k_params=s["pk"], cache_v_params=s["pv"], block_table=s["table"])
        if op == "attend":
            B.prefill_attn_varlen_cache4(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["ck"], s["cv"], s["offsets"],
                                         s["out"], s["lse"], scale=s["scale"], window=s["case"]["window"], **cache)
        elif op == "write":
            B.prefill_attn_cache4_write(s["k"], s["v"], s["cu_q"], s["ck"], s["cv"], s["offsets"], **cache)
        B.prefill_attn_cache4_read(s["ck"], s["cv"], s["cu_q"], s["offsets"], s["k_back"], s["v_back"], **cache)
    got = {"k": s["k_back"], "v": s["v_back"]}                        # the call's rows as the values they stand for
    if op == "attend":
        got.update(out=s["out"], lse=s["lse"])
    if op != "read":
        got.update(k_params=s["pk"], v_params=s["pv"])                # the scales and minima of the whole cache
    return got


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence and one KV head at a time
# ---------------------------------------------------------------------------

def _rows64(s, which, b, h, lo, hi):
    """Values of the cache rows of positions [lo, hi) of sequence b and KV head h."""
    pos = torch.arange(lo, hi, device=DEV)
    slot, row = torch.full_like(pos, b), pos
    if s["table"] is not None:
        slot, row = s["table"][b].long()[pos // s["case"]["block"]], pos % s["case"]["block"]
    codes, params = s["c" + which][slot, h, row].int(), s["p" + which][slot, h, row].double()
    d = s["case"]["dim"]
    out = torch.empty((hi - lo, d), dtype=torch.float64, device=DEV)
    for ch in range(d):
        code = (codes[:, ch // 2] >> (4 * (ch % 2))) & 15
        out[:, ch] = code * params[:, ch // s["case"]["group"], 0] + params[:, ch // s["case"]["group"], 1]
    return out


def _stored64(x, group):
    """What rows x [..., d] stand for once they are stored (the format's roundings to 32 and 16 bits kept)."""
    out = torch.empty(x.shape, dtype=torch.float64, device=DEV)
    for g0 in range(0, x.shape[-1], group):
        y = x[..., g0:g0 + group].double()
        lo, hi = y.min(-1, keepdim=True).values, y.max(-1, keepdim=True).values
        fifteenth = float(torch.tensor(1.0 / 15.0, dtype=torch.float32))
        s = ((hi - lo).float().double() * fifteenth).float().to(torch.bfloat16).double()
        s = torch.where(s < 2.0 ** -126, 0.0, s)
        r = torch.where(s > 0, (1.0 / s).float().double(), 0.0)
        code = ((y - lo).float().double() * r).float().double().round().clamp(max=15.0)
        out[..., g0:g0 + group] = lo + code * s
    return out


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    new, ctx = _lengths(c)
    H, Hk, d = c["heads"], c["kv_heads"], c["dim"]
    G = H // Hk
    stored = {"k": _stored64(s["k"], c["group"]), "v": _stored64(s["v"], c["group"]), "k_params": None, "v_params": None}
    if c["op"] == "write":
        return stored
    if c["op"] == "read":
        out = {w: torch.empty((s["T"], Hk, d), dtype=torch.float64, device=DEV) for w in ("k", "v")}
        for w in ("k", "v"):
            t0 = 0
            for b, (n, p) in enumerate(zip(new, ctx)):
                for h in range(Hk):
                    out[w][t0:t0 + n, h] = _rows64(s, w, b, h, p, p + n)
                t0 += n
        return out
    window, scale = c["window"], s["scale"]
    if H * sum(n * min(p + n, window + 512 if window else p + n) for n, p in zip(new, ctx)) * d > 1 << 41:
        return None
    out = torch.zeros((s["T"], H, d), dtype=torch.float64, device=DEV)
    lse = torch.zeros((s["T"], H), dtype=torch.float64, device=DEV)
    for h in range(Hk):
        t0 = 0
        for b, (n, p) in enumerate(zip(new, ctx)):
            k = torch.cat([_rows64(s, "k", b, h, 0, p), s["k"][t0:t0 + n, h].double()])
            v = torch.cat([_rows64(s, "v", b, h, 0, p), s["v"][t0:t0 + n, h].double()])
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                first = max(0, p + i0 - window + 1) if window else 0
                j = torch.arange(first, p + i1, device=DEV)
                at = torch.arange(p + i0, p + i1, device=DEV)[:, None]
                see = j <= at
                if window:
                    see &= at - j < window
                q = s["q"][t0 + i0:t0 + i1, h * G:(h + 1) * G].double()
                x = torch.einsum("igd,jd->igj", q, k[first:p + i1]) * scale
                x = torch.where(see[:, None], x, -math.inf)
                z = torch.logsumexp(x, -1)
                e = torch.exp(x - z[..., None])
                out[t0 + i0:t0 + i1, h * G:(h + 1) * G] = torch.einsum("igj,jd->igd", e, v[first:p + i1])
                lse[t0 + i0:t0 + i1, h * G:(h + 1) * G] = z
            t0 += n
    return {"out": out, "lse": lse, **stored}
