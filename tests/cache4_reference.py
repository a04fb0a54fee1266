"""Plain 64-bit forms of the 4-bit cache's calls, and the error bounds their tests use.

A rounding to bf16 is off by at most u = 2^-8 of the value, one to fp16 by 2^-11, one to fp32 by 2^-24.

Attention.  Let P be the exact softmax weights, s, m, c a cached key's or value's scale, minimum and code.

The row kernel rounds p s to fp16 ahead of the product with c, and a new token's p to bf16 ahead of the
product with its value, so O is off by at most  sum_j P_j a_j,  a_j = 2^-11 s_j c_j for a cached key and
u |v_j| for a new one.  Weights are scaled so that a row's largest is at least 2^7: those below fp16's normal
range are off by 2^-25 absolutely, 2^-32 of the largest p s, 15 times as much in O, each.

The tile kernel's cached keys are sums of two bf16 terms, off by at most 2^-16, which is as much of
scale sum_i |q_i| |k_i| in a score.  Cached values and their p are rounded to fp16, 2^-11 each, where a tile's values
are within its range, else to bf16 like a new token's p; values below 2^-14 are off by 2^-25.  A bound of a call
says which (halves); weights below 2^-14 are 2^-21 of the largest at least, off by 2^-32 of it.

Both round out once.  fp32: a score is a sum of d / 16 products of 16 channels and d / 32 parameter terms,
each sum off by at most 2^-22 of what it sums up: together 2^-18 of A = scale sum_i |q_i| (|m_i| + c_i s_i), which
covers its product with the scale and the difference to the maximum too.  Exponentials and sums add 2^-18 of
the weights, and O's sums 2^-18 of  sum_j P_j (|m_j| + c_j s_j).  A score off by x moves every P by a factor within e^(+-2x).
"""
import math

import torch

U = 2.0 ** -8


def quantise(x, group):
    """(codes uint8 [..., d / 2], params bf16 [..., d / group, 2]) of bf16 rows x, by the format's steps in fp32."""
    y = x.float().unflatten(-1, (-1, group))
    lo, hi = y.amin(-1) + 0.0, y.amax(-1)                     # (0 for -0)
    s = ((hi - lo) * torch.tensor(1.0 / 15.0)).to(torch.bfloat16)
    s = torch.where(s.float() >= 2.0 ** -126, s, torch.zeros_like(s))
    r = torch.where(s > 0, torch.ones(()) / s.float(), torch.zeros(()))
    c = torch.round((y - lo[..., None]) * r[..., None]).clamp(max=15).to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack([s, lo.to(torch.bfloat16)], -1)


def split(codes, params):
    """(codes, scales, minima) of rows, each [..., d] in 64 bits."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double()
    p = params.double().repeat_interleave(c.shape[-1] // params.shape[-2], -2)
    return c, p[..., 0], p[..., 1]


def values(codes, params):
    c, s, m = split(codes, params)
    return m + c * s


class Cache:
    """A 4-bit cache on the CPU: contiguous slots, or pools with a block table in random order (block > 0)."""

    def __init__(self, g, seqs, cap, hk, d, group, block=0, spare=3, kind="normal"):
        self.seqs, self.cap, self.hk, self.d, self.group, self.block = seqs, cap, hk, d, group, block
        self.table, slots, rows = None, seqs, cap
        if block:
            per = -(-cap // block)
            self.cap = per * block
            order = torch.randperm(seqs * per + spare, generator=g)
            self.table = order[:seqs * per].reshape(seqs, per).to(torch.int32)
            slots, rows = seqs * per + spare, block
        self.codes, self.params = [], []
        offset = 2 * torch.randn((1, hk, 1, d), generator=g)
        for which in range(2):
            x = torch.randn((slots, hk, rows, d), generator=g) + (offset if which == 0 else 0)
            if kind == "large":
                x *= 2.0 ** 60
            c, p = quantise(x.to(torch.bfloat16), group)
            self.codes.append(c)
            self.params.append(p)

    def at(self, b, pos):
        """(slot, row) of positions of sequence b."""
        if self.table is None:
            return torch.full_like(pos, b), pos
        return self.table[b].long()[pos // self.block], pos % self.block

    def rows(self, which, b, h, n, lo=0):
        """(codes, params) of positions [lo, n)."""
        slot, row = self.at(b, torch.arange(lo, n))
        return self.codes[which][slot, h, row], self.params[which][slot, h, row]

    def spoil(self, lens):
        """Fills every parameter past a sequence's length with NaN (nothing reads them)."""
        for p in self.params:
            keep = torch.zeros(p.shape[0], p.shape[2], dtype=torch.bool)
            for b, n in enumerate(lens):
                keep[self.at(b, torch.arange(n))] = True
            p.permute(0, 2, 1, 3, 4)[~keep] = math.nan

    def stored(self, k, v, cu, lens):
        """(codes, params) of the cache after the packed rows went in at positions lens[b] ..."""
        codes, params = [x.clone() for x in self.codes], [x.clone() for x in self.params]
        for which, x in enumerate((k, v)):
            c, p = quantise(x, self.group)
            for b, at in enumerate(lens):
                n = cu[b + 1] - cu[b]
                slot, row = self.at(b, torch.arange(at, at + n))
                codes[which][slot, :, row] = c[cu[b]:cu[b + 1]]
                params[which][slot, :, row] = p[cu[b]:cu[b + 1]]
        return codes, params


def rotate(x, pos, theta):
    """Rotary embedding of x [n, heads, d] at positions pos, rounded to bf16 (fp32 steps as documented)."""
    half = x.shape[-1] // 2
    inv = (1.0 / torch.pow(torch.tensor(theta, dtype=torch.float32), torch.arange(half) * 2.0 / x.shape[-1]))
    a = (pos.float()[:, None] * inv).double()
    c, s = torch.cos(a)[:, None], torch.sin(a)[:, None]
    lo, hi = x[..., :half].double(), x[..., half:].double()
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def attention(cache, q, k, v, cu, lens, scale, causal=True, window=0, tiles=False, halves=True):
    """(out, lse, bound on out's error, bound on lse's) in 64 bits.  tiles: the bounds of the tile kernel too; halves:
    every tile's cached values are within fp16's range."""
    t, heads, d = q.shape
    hk = k.shape[1]
    g = heads // hk
    out, bound = torch.zeros((t, heads, d), dtype=torch.float64), torch.zeros((t, heads, d), dtype=torch.float64)
    lse, lbound = torch.zeros((t, heads), dtype=torch.float64), torch.zeros((t, heads), dtype=torch.float64)
    for b, p in enumerate(lens):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        pos = p + torch.arange(n)[:, None]
        j = torch.arange(p + n)
        see = (j <= pos) if causal else torch.ones((n, p + n), dtype=torch.bool)
        if window:
            see = see & (j > pos - window)
        for h in range(hk):
            kc, ks, km = split(*cache.rows(0, b, h, p))
            vc, vs, vm = split(*cache.rows(1, b, h, p))
            kn, vn = k[rows, h].double(), v[rows, h].double()
            kk, kparts = torch.cat([km + kc * ks, kn]), torch.cat([km.abs() + kc * ks, kn.abs()])
            val, vparts = torch.cat([vm + vc * vs, vn]), torch.cat([vm.abs() + vc * vs, vn.abs()])
            step = torch.cat([2.0 ** -11 * vc * vs, U * vn.abs()])
            least = torch.cat([vs, torch.zeros_like(vn)])
            qq = q[rows, h * g:(h + 1) * g].double()
            x = torch.einsum("igd,jd->igj", qq, kk) * scale
            x = torch.where(see[:, None], x, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[..., None])
            ab = torch.einsum("igd,jd->igj", qq.abs(), kk.abs()) * scale
            parts = torch.einsum("igd,jd->igj", qq.abs(), kparts) * scale
            x_err = parts * 2.0 ** -18 + (ab * 2.0 ** -16 if tiles else 0.0) + 2.0 ** -18
            ex = torch.where(see[:, None], x_err, 0.0).amax(-1)
            o = torch.einsum("igj,jd->igd", w, val)
            mean = torch.einsum("igj,jd->igd", w, val.abs())
            r = torch.einsum("igj,jd->igd", w, step) + 2.0 ** -18 * torch.einsum("igj,jd->igd", w, vparts)
            r = r + 15 * 2.0 ** -32 * (p + n) * (w[..., None] * least).amax(2)
            if tiles and halves:
                fine = torch.where(j[:, None] < p, 2 * 2.0 ** -11 * val.abs() + 2.0 ** -25, U * val.abs())
                r = r + torch.einsum("igj,jd->igd", w, fine) + 2.0 ** -32 * (p + n) * val.abs().amax() * w.amax(-1)[..., None]
            elif tiles:
                r = r + 2 * U * mean
            out[rows, h * g:(h + 1) * g] = o
            lse[rows, h * g:(h + 1) * g] = z
            grown = torch.expm1(2 * ex)[..., None] * mean
            # out itself may be off by what precedes its own rounding
            err = r * (1 + torch.expm1(2 * ex)[..., None]) + grown
            bound[rows, h * g:(h + 1) * g] = err + U * (o.abs() + err)
            lbound[rows, h * g:(h + 1) * g] = ex + z.abs() * 2.0 ** -20 + 2.0 ** -20
    return out, lse, bound, lbound
