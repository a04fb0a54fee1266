"""Plain 64-bit forms of the long-context operators, and the caches their tests use.

Everything here is elementary torch on the CPU in float64, one sequence and one
KV head at a time, written from the definitions:

  visible(p, j): j <= p (causal) and (no window, or j > p - W, or j < sinks)
  out_i = sum_j softmax_j(scale q_i . k_j) v_j,  lse_i = log sum_j exp(scale q_i . k_j)
  weight_j = sum_i exp(scale q_i . k_j - lse_i)

Tolerances.  The kernels round P (and int8 values) to bf16 before P V and the
output once at the end; a rounding to bf16 is off by at most 2^-8 of the value.
With A = sum_j p_j |v_j| / l the output is within
    2^-8 (A + |out|)  (+ 2^-8 A for int8 values)  + SCORE * A,
where SCORE = 2^-11 bounds twice the error of a score: fp32 accumulation of d =
128 products, each sum off by at most d * 2^-23 * sum |q k| * scale, about 1.1e-4
for sum |q k| * scale <= 7.3 (N(0, 1) data), on numerator and denominator.  The
lse moves by one score error at most, and a key weight by 2^-11 of itself.
"""
import math

import torch

BF16 = 2.0 ** -8
SCORE = 2.0 ** -11


class Cache:
    """A bf16 or int8 cache, contiguous or paged, with its logical contents.

    k[b], v[b]: float64 [n_kv_heads, P_b, d], what the cached rows stand for.
    Rows that hold nothing are filled with NaN (bf16) or NaN scales (int8).
    """

    def __init__(self, g, lens, cap, n_kv_heads, d, block=0, int8=False, prefix=0):
        self.lens, self.cap, self.hk, self.d, self.block, self.int8 = lens, cap, n_kv_heads, d, block, int8
        b = len(lens)
        self.table = self.prefix_table = None
        if block:
            nb = -(-cap // block)
            self.cap = nb * block
            npre = -(-prefix // block)
            order = torch.randperm(b * nb + npre + 3, generator=g).to(torch.int32)
            self.table = order[:b * nb].reshape(b, nb).contiguous()
            self.prefix_table = order[b * nb:b * nb + npre].contiguous()
            shape = (b * nb + npre + 3, n_kv_heads, block, d)
        else:
            shape = (b, n_kv_heads, cap, d)
        self.shape = shape
        self.data, self.scale = [], []
        for _ in range(2):
            if int8:
                self.data.append(torch.randint(-127, 128, shape, generator=g, dtype=torch.int32).to(torch.int8))
                self.scale.append(torch.full(shape[:-1], math.nan))
            else:
                self.data.append(torch.full(shape, math.nan, dtype=torch.bfloat16))
                self.scale.append(None)
        for i, n in enumerate(lens):
            self.fill(g, lambda pos, i=i: self.at(i, pos), n)
        # the shared prefix: pool blocks of a paged cache, tensors of its own otherwise
        self.prefix, self.pre_data, self.pre_scale = prefix, [None, None], [None, None]
        if prefix and block:
            self.fill(g, lambda pos: (self.prefix_table.long()[pos // block], pos % block), prefix)
        elif prefix:
            cap = prefix + 5
            for w in range(2):
                x, s = self.values(g, prefix)
                pad = torch.full((n_kv_heads, cap, d), math.nan, dtype=torch.bfloat16) if not int8 else \
                    torch.zeros((n_kv_heads, cap, d), dtype=torch.int8)
                pad[:, :prefix] = x
                self.pre_data[w] = pad
                if int8:
                    self.pre_scale[w] = torch.full((n_kv_heads, cap), math.nan)
                    self.pre_scale[w][:, :prefix] = s

    def values(self, g, n):
        if not self.int8:
            return torch.randn((self.hk, n, self.d), generator=g).to(torch.bfloat16), None
        x = torch.randint(-127, 128, (self.hk, n, self.d), generator=g, dtype=torch.int32).to(torch.int8)
        return x, torch.rand((self.hk, n), generator=g) * 0.012 + 0.008

    def fill(self, g, where, n):
        if n == 0:
            return
        slot, row = where(torch.arange(n))
        for w in range(2):
            x, s = self.values(g, n)
            self.data[w][slot, :, row] = x.transpose(0, 1)
            if self.int8:
                self.scale[w][slot, :, row] = s.T

    def at(self, b, pos):
        """(slot or block, row) of positions pos (a tensor) of sequence b."""
        if not self.block:
            return torch.full_like(pos, b), pos
        return self.table[b].long()[pos // self.block], pos % self.block

    def logical(self, w, b, n=None):
        """float64 [n_kv_heads, n, d] of sequence b (w = 0: keys, 1: values)."""
        slot, row = self.at(b, torch.arange(self.lens[b] if n is None else n))
        x = self.data[w][slot, :, row].double()
        if self.int8:
            x = x * self.scale[w][slot, :, row].double()[..., None]
        return x.transpose(0, 1)

    def logical_prefix(self, w):
        if not self.prefix:
            return torch.zeros((self.hk, 0, self.d), dtype=torch.float64)
        if self.block:
            pos = torch.arange(self.prefix)
            slot, row = self.prefix_table.long()[pos // self.block], pos % self.block
            x = self.data[w][slot, :, row].double()
            if self.int8:
                x = x * self.scale[w][slot, :, row].double()[..., None]
            return x.transpose(0, 1)
        x = self.pre_data[w][:, :self.prefix].double()
        return x if not self.int8 else x * self.pre_scale[w][:, :self.prefix].double()[..., None]

    def written(self, w, new, cu):
        """The cache image after the new rows new [T, hk, d] (bf16) were written: (data, scale)."""
        data = self.data[w].clone()
        scale = None if self.scale[w] is None else self.scale[w].clone()
        for b, p in enumerate(self.lens):
            n = cu[b + 1] - cu[b]
            slot, row = self.at(b, torch.arange(p, p + n))
            x = new[cu[b]:cu[b + 1]]
            if self.int8:
                f = x.float()
                s = f.abs().amax(-1) / 127.0
                x = torch.where(s[..., None] > 0, (f / s[..., None]).round().clamp(-127, 127), 0.0).to(torch.int8)
                scale[slot, :, row] = s
            data[slot, :, row] = x
        return data, scale


def bits(t):
    """Bit image of a tensor, so that NaN sentinels compare."""
    return t.contiguous().view({1: torch.int8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def rotate(x, pos, theta):
    """Rotary embedding (rotate-half) of bf16 x [n, h, d] at positions pos, rounded to bf16 like the library's."""
    if not theta:
        return x
    half = x.shape[-1] // 2
    inv = (1.0 / torch.tensor(theta, dtype=torch.float32) ** (torch.arange(half, dtype=torch.float32) * 2 / x.shape[-1]))
    ang = (pos.float()[:, None] * inv).double()[:, None]
    a, b = x[..., :half].double(), x[..., half:].double()
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).to(torch.bfloat16)


def sequences(cache, q, k, v, new, theta=0.0):
    """Per sequence: (token range, q, k of the new tokens as attention sees them, v)."""
    cu = cumulative(new)
    for b, n in enumerate(new):
        t = slice(cu[b], cu[b + 1])
        pos = torch.arange(n) + cache.prefix + cache.lens[b]
        yield b, t, rotate(q[t], pos, theta), rotate(k[t], pos, theta), None if v is None else v[t]


def visible(p, n, causal, window, sinks):
    """[n, p + n]: does the query at position p + i see key j."""
    i, j = torch.arange(p, p + n)[:, None], torch.arange(p + n)
    if not causal:
        return torch.ones((n, p + n), dtype=torch.bool)
    see = j <= i
    return see & ((i - j < window) | (j < sinks)) if window else see


def attention(cache, q, k, v, new, scale, causal=True, window=0, sinks=0, theta=0.0):
    """(out, lse, A) in float64, A = sum_j p_j |v_j| per output element."""
    h, g = q.shape[1], q.shape[1] // cache.hk
    out = torch.zeros(q.shape, dtype=torch.float64)
    mag, lse = torch.zeros_like(out), torch.zeros((q.shape[0], h), dtype=torch.float64)
    pre = [cache.logical_prefix(w) for w in range(2)]
    for b, t, qb, kb, vb in sequences(cache, q, k, v, new, theta):
        n, p = qb.shape[0], cache.lens[b]
        if n == 0:
            continue
        see = torch.cat([torch.ones((n, cache.prefix), dtype=torch.bool), visible(p, n, causal, window, sinks)], 1)
        keys = torch.cat([pre[0], cache.logical(0, b), kb.double().transpose(0, 1)], 1)
        vals = torch.cat([pre[1], cache.logical(1, b), vb.double().transpose(0, 1)], 1)
        for i in range(h):
            x = (qb[:, i].double() @ keys[i // g].T) * scale
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, -1)
            w = torch.exp(x - z[:, None])
            out[t, i], mag[t, i], lse[t, i] = w @ vals[i // g], w @ vals[i // g].abs(), z
    return out, lse, mag


def key_weights(cache, q, k, new, lse, scale, old, causal=True, window=0, sinks=0, theta=0.0):
    """The weights after the call, float64, laid out like the cache's rows."""
    h, g = q.shape[1], q.shape[1] // cache.hk
    got = old.double().clone()
    for b, t, qb, kb, _ in sequences(cache, q, k, None, new, theta):
        n, p = qb.shape[0], cache.lens[b]
        if n == 0:
            continue
        see = visible(p, n, causal, window, sinks)
        keys = torch.cat([cache.logical(0, b), kb.double().transpose(0, 1)], 1)
        add = torch.zeros((cache.hk, p + n), dtype=torch.float64)
        for i in range(h):
            x = (qb[:, i].double() @ keys[i // g].T) * scale - lse[t, i].double()[:, None]
            add[i // g] += torch.exp(x).masked_fill(~see, 0.0).sum(0)
        slot, row = cache.at(b, torch.arange(p))
        got[slot, :, row] += add[:, :p].T
        slot, row = cache.at(b, torch.arange(p, p + n))
        got[slot, :, row] = add[:, p:].T
    return got


def evicted(w, budget, sinks, recent):
    """Kept positions of one head's weights w (a 1-D tensor), ascending."""
    n = w.numel()
    if n <= budget:
        return torch.arange(n)
    mid = [(0 if math.isnan(x) else 1, -x if not math.isnan(x) else 0.0, i + sinks)
           for i, x in enumerate(w[sinks:n - recent].tolist())]
    best = sorted(i for _, _, i in sorted(mid)[:budget - sinks - recent])
    return torch.tensor(list(range(sinks)) + best + list(range(n - recent, n)), dtype=torch.long)
