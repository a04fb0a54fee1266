"""GPU tests of the 4-bit cache: attention over it, writing it and reading it back, each against its plain 64-bit
form (tests/cache4_reference.py, where the bounds are derived)."""
import concurrent.futures
import math

import pytest
import torch

from prefill_phase_attention_gb300 import binding
from tests import cache4_reference as R

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from prefill_phase_attention_gb300 import build
    build.build()
    binding.load()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")


def cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def guarded(x):
    """(buffer with bands on both sides, the view that holds x)."""
    n = x.numel() * x.element_size()
    buf = torch.full((n + 2 * GUARD,), 0x5a, dtype=torch.uint8, device="cuda")
    view = buf[GUARD:GUARD + n].view(x.dtype).view(x.shape)
    view.copy_(x)
    return buf, view


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8).cpu(), b.contiguous().view(torch.uint8).cpu())


class Call:
    """Inputs of one call on the CPU, their GPU copies, and what is written in guarded buffers."""

    def __init__(self, seed, new, lens, d=128, hk=2, share=2, group=None, block=0, kind="normal", slack=3, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.d, self.hk, self.share = new, lens, d, hk, share
        cap = max(p + n for p, n in zip(lens, new)) + slack
        self.cache = R.Cache(g, len(new), cap, hk, d, group or d, block, kind=kind)
        t = sum(new) + pad
        size = 2.0 ** 60 if kind == "large" else 1.0
        self.q = (torch.randn((t, hk * share, d), generator=g) / size).to(torch.bfloat16)
        self.k = (torch.randn((t, hk, d), generator=g) * size).to(torch.bfloat16)
        self.v = (torch.randn((t, hk, d), generator=g) * size).to(torch.bfloat16)
        self.cu, self.scale = cumulative(new), d ** -0.5
        self.meta = (i32(self.cu), i32(cumulative([p + n for p, n in zip(lens, new)])))
        self.offsets = i32(lens)
        self.dev = [x.cuda() for x in (self.q, self.k, self.v)]
        self.cache.spoil(lens)
        self.codes = [guarded(x) for x in self.cache.codes]
        self.params = [guarded(x) for x in self.cache.params]
        self.out = guarded(torch.full(self.q.shape, math.nan, dtype=torch.bfloat16))
        self.lse = guarded(torch.full((t, hk * share), math.nan))
        self.opts = dict(cache_k_params=self.params[0][1], cache_v_params=self.params[1][1],
                         block_table=None if self.cache.table is None else self.cache.table.cuda())

    def attend(self, **kw):
        binding.prefill_attn_varlen_cache4(*self.dev, *self.meta, self.codes[0][1], self.codes[1][1], self.offsets,
                                           self.out[1], self.lse[1], scale=self.scale, **self.opts, **kw)
        self.expanded = binding.load().prefill_attn_last_schedule() != 0  # (the row kernel has no schedule)

    def write(self, **kw):
        binding.prefill_attn_cache4_write(*self.dev[1:], self.meta[0], self.codes[0][1], self.codes[1][1], self.offsets,
                                          **self.opts, **kw)

    def guards(self):
        for buf, _ in self.codes + self.params + [self.out, self.lse]:
            assert (buf[:GUARD] == 0x5a).all() and (buf[-GUARD:] == 0x5a).all(), "write outside a buffer"

    def check_cache(self, k=None):
        codes, params = self.cache.stored(self.k if k is None else k, self.v, self.cu, self.lens)
        for which in range(2):
            assert same_bits(self.codes[which][1], codes[which]), "codes"
            assert same_bits(self.params[which][1], params[which]), "parameters"

    def check(self, causal=True, window=0, tiles=False, halves=True):
        torch.cuda.synchronize()
        assert binding.prefill_attn_device_status() == 0
        out, lse, bound, lbound = R.attention(self.cache, self.q, self.k, self.v, self.cu, self.lens, self.scale, causal,
                                              window, tiles, halves)
        t = self.cu[-1]
        assert self.out[1][t:].isnan().all() and self.lse[1][t:].isnan().all(), "rows behind the last sequence"
        got, glse = self.out[1][:t].double().cpu(), self.lse[1][:t].double().cpu()
        out, lse, bound, lbound = out[:t], lse[:t], bound[:t], lbound[:t]
        assert got.isfinite().all() and glse.isfinite().all()
        assert ((got - out).abs() <= bound).all(), ((got - out).abs() / bound).max()
        assert ((glse - lse).abs() <= lbound).all(), ((glse - lse).abs() / lbound).max()
        self.check_cache()
        self.guards()


DIMS = [(128, 128), (128, 64), (128, 32), (64, 64), (64, 32), (32, 32)]


@pytest.mark.parametrize("block", [0, 8, 16, 128])
@pytest.mark.parametrize("d,group", DIMS)
def test_decode_rows(d, group, block):
    c = Call(1, [1] * 9, [0, 1, 31, 32, 33, 255, 256, 257, 1000], d, group=group, block=block, share=4)
    c.attend()
    c.check()


@pytest.mark.parametrize("hk,share", [(1, 1), (1, 8), (3, 5), (2, 16), (1, 48), (1, 128), (8, 1)])
def test_head_layouts(hk, share):
    c = Call(2, [1, 2, 1], [77, 500, 3], hk=hk, share=share, group=32)
    c.attend()
    c.check()


@pytest.mark.parametrize("d,group", [(128, 64), (64, 64), (32, 32)])
@pytest.mark.parametrize("new,lens", [([5, 1, 7], [100, 2000, 0]), ([9, 17, 1, 0], [31, 33, 64, 9]), ([8, 16], [0, 257])])
def test_drafts(d, group, new, lens):
    for block in (0, 16):
        c = Call(3, new, lens, d, group=group, block=block, share=3)
        c.attend()
        c.check()


@pytest.mark.parametrize("block", [0, 8, 128])
@pytest.mark.parametrize("d,group", DIMS)
def test_chunks(d, group, block):
    """Chunks long enough for the tile kernel, decode rows and drafts beside them."""
    c = Call(11, [300, 1, 129, 4, 0, 200], [0, 500, 127, 33, 9, 260], d, hk=1, group=group, block=block, share=16)
    c.attend()
    assert c.expanded
    c.check(tiles=True)


@pytest.mark.parametrize("new,past,hk,share", [(9, 200, 2, 4), (40, 3, 1, 1), (64, 128, 1, 3), (513, 1000, 4, 4), (130, 0, 3, 16),
                                               (257, 129, 2, 1), (300, 200, 8, 1), (70, 250, 1, 48), (40, 100, 1, 128)])
@pytest.mark.parametrize("block", [0, 32])
def test_one_chunk(new, past, hk, share, block):
    c = Call(12, [new], [past], hk=hk, share=share, group=64, block=block)
    c.attend()
    c.check(tiles=c.expanded)


def test_more_long_chunks_than_the_pool_holds():
    """The 1 GiB of expanded blocks holds one of these three sequences; the others go through the row kernel.  Each
    alone has the tile kernel: both ways agree within their bounds.  (Every sequence's 131000 cached positions
    are 64 blocks of the pool over and over.)"""
    g = torch.Generator().manual_seed(17)
    hk, d, bs, p, n, b = 8, 128, 16, 131000, 400, 3
    per = -(-(p + n) // bs)
    fresh = per - p // bs                                        # blocks that the new tokens go to
    cache = R.Cache(g, 1, (64 + b * fresh) * bs, hk, d, 128, bs, spare=0)
    table = torch.randint(0, 64, (b, per), generator=g)
    table[:, -fresh:] = 64 + torch.arange(b * fresh).reshape(b, fresh)
    table = table.to(torch.int32).cuda()
    codes, params = [x.cuda() for x in cache.codes], [x.cuda() for x in cache.params]
    q, k, v = ((torch.randn((b * n, hk, d), generator=g) * s).to(torch.bfloat16).cuda() for s in (3, 1, 1))

    def attend(rows, seqs):
        out, m = torch.empty_like(q[rows]), len(seqs)
        cu, cu_k = i32([n * i for i in range(m + 1)]), i32([(n + p) * i for i in range(m + 1)])
        c = [x.clone() for x in codes + params]
        binding.prefill_attn_varlen_cache4(q[rows], k[rows], v[rows], cu, cu_k, c[0], c[1], i32([p] * m), out,
                                           cache_k_params=c[2], cache_v_params=c[3], block_table=table[seqs].contiguous())
        torch.cuda.synchronize()
        assert binding.prefill_attn_device_status() == 0
        return out.double(), c

    together, c = attend(slice(0, b * n), [0, 1, 2])
    largest = max(v.double().abs().max(), R.values(cache.codes[1], cache.params[1]).abs().max())
    for i in range(b):
        alone, e = attend(slice(i * n, (i + 1) * n), [i])
        # off by 2 u (values, p) and 2^-11 (p s) of the largest value, new tokens' weights by u, and each out's own rounding u
        assert ((together[i * n:(i + 1) * n] - alone).abs() <= 6 * R.U * largest).all()
        blocks = table[i, -fresh:].long()
        for x, y in zip(c, e):
            assert same_bits(x[blocks], y[blocks])


@pytest.mark.parametrize("new,pad", [([1, 3], 7), ([5], 600), ([130], 70), ([0], 300), ([300, 1, 129], 200), ([2, 3, 1], 900)])
def test_rows_behind_the_last_sequence(new, pad):
    """What a replayed call over fewer tokens than it was captured for has: they are left as they were."""
    c = Call(18, new, [100, 257, 31][:len(new)], share=8, group=64, pad=pad)
    c.attend()
    c.check(tiles=c.expanded)
    w = Call(19, new, [100, 257, 31][:len(new)], group=64, pad=pad)
    w.write()
    w.check_cache()
    k = torch.full(w.k.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    binding.prefill_attn_cache4_read(w.codes[0][1], w.codes[1][1], w.meta[0], w.offsets, k, v, **w.opts)
    t = w.cu[-1]
    for got, x in ((k, w.k), (v, w.v)):
        assert got[t:].isnan().all()
        assert same_bits(got[:t], R.values(*R.quantise(x[:t], 64)).float().to(torch.bfloat16))


@pytest.mark.parametrize("window", [1, 100, 128, 300])
@pytest.mark.parametrize("block", [0, 16])
def test_chunks_under_windows(window, block):
    c = Call(13, [460, 1, 150], [400, 300, 10], hk=1, share=16, group=32, block=block)
    c.attend(window=window)
    assert c.expanded
    c.check(window=window, tiles=True)


@pytest.mark.parametrize("window,past", [(129, 1000), (130, 1024), (257, 1025), (385, 1151), (5000, 1023)])
def test_one_chunk_under_a_window(window, past):
    c = Call(16, [200], [past], hk=1, share=16, group=64, block=32)
    c.attend(window=window)
    assert c.expanded
    c.check(window=window, tiles=True)


@pytest.mark.parametrize("block", [0, 16])
def test_chunks_over_values_of_any_size(block):
    """Tiles whose values are outside fp16's range (large, or all tiny) beside such as are inside it, in each sequence."""
    c = Call(15, [300, 129, 400], [700, 129, 128], d=64, hk=1, share=16, group=32, block=block)
    slots = torch.arange(c.cache.codes[1].shape[0])
    size = torch.exp2(torch.tensor([0.0, 20.0, -20.0, 90.0, -9.0])[slots % 5 if block else slots % 2 * 2])
    x = c.cache.params[1].double() * size[:, None, None, None, None]
    if not block:
        x[0, :, 200:400] *= 2.0 ** 30
        x[2, :, :1] *= 2.0 ** 30
    c.cache.params[1] = x.to(torch.bfloat16)
    c.params[1][1].copy_(c.cache.params[1])
    c.attend()
    assert c.expanded
    c.check(tiles=True, halves=False)


def test_chunks_with_all_keys_visible():
    c = Call(14, [460, 1, 150], [100, 300, 10], hk=1, share=16, group=128)
    c.attend(causal=False)
    assert c.expanded
    c.check(causal=False, tiles=True)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 100, 5000])
@pytest.mark.parametrize("block", [0, 16])
def test_windows(window, block):
    c = Call(4, [1, 3, 1, 12], [1000, 257, 5, 40], group=64, block=block)
    c.attend(window=window)
    c.check(window=window)


def test_all_keys_visible():
    c = Call(5, [4, 1, 11], [64, 33, 0], group=32)
    c.attend(causal=False)
    c.check(causal=False)


def test_one_long_row():
    """Every CTA has a share of the same rows."""
    c = Call(6, [1], [40000], hk=1, share=4)
    c.attend()
    c.check()


def test_many_sequences():
    """More sequences than a CTA keeps in shared memory."""
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(0, 70, (700,), generator=g).tolist()
    new = torch.randint(0, 3, (700,), generator=g).tolist()
    c = Call(7, new, lens, d=32, hk=1, share=2)
    c.attend()
    c.check()


@pytest.mark.parametrize("new,lens", [([1, 6], [300, 45]), ([3, 1, 9], [0, 0, 0])])
def test_large_values(new, lens):
    """Keys and values (and their scales) far outside fp16's range."""
    c = Call(8, new, lens, group=64, kind="large")
    c.attend()
    c.check()


@pytest.mark.parametrize("new", [[1, 1, 1], [3, 2, 60]])
def test_values_of_very_different_size(new):
    """Rows of V whose scales differ by 2^60, and queries so large that the weights differ as much: what a row adds
    may be the product of a tiny weight and a huge value."""
    c = Call(15, new, [600, 64, 40], group=64)
    g = torch.Generator().manual_seed(1)
    for which in range(2):
        size = torch.randint(-30, 31, c.cache.params[1].shape[:3], generator=g).double()
        if which == 0:
            size *= 0.1
        x = c.cache.params[which].double() * torch.exp2(size)[..., None, None]
        c.cache.params[which] = x.to(torch.bfloat16)
        c.params[which][1].copy_(c.cache.params[which])
    c.q *= 6
    c.dev[0].copy_(c.q)
    c.attend()
    c.check(tiles=max(new) > 16, halves=False)


@pytest.mark.parametrize("new", [[1, 3], [1100, 1]])
def test_pools_past_4_gib(new):
    """Blocks whose codes begin past 2^32 bytes: the same bits as in a small pool."""
    c = Call(70, new, [700, 40], hk=8, share=1, block=16)
    blocks = 2 ** 32 // (8 * 16 * 64) + 5
    small = [x[1].clone() for x in c.codes + c.params]
    big = [torch.empty((blocks + x.shape[0], *x.shape[1:]), dtype=x.dtype, device="cuda") for x in small]
    for x, y in zip(big, small):
        x[blocks:] = y
    c.attend()
    out, lse = c.out[1].clone(), c.lse[1].clone()
    c.opts.update(cache_k_params=big[2], cache_v_params=big[3], block_table=c.opts["block_table"] + blocks)
    c.codes[:2] = [(None, big[0]), (None, big[1])]
    c.attend()
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == 0
    assert same_bits(c.out[1], out) and same_bits(c.lse[1], lse)
    codes, params = c.cache.stored(c.k, c.v, c.cu, c.lens)
    for which in range(2):
        assert same_bits(big[which][blocks:], codes[which]) and same_bits(big[2 + which][blocks:], params[which])
    k, v = torch.empty_like(c.dev[1]), torch.empty_like(c.dev[2])
    c.write()
    binding.prefill_attn_cache4_read(big[0], big[1], c.meta[0], c.offsets, k, v, **c.opts)
    for which, (got, x) in enumerate(((k, c.k), (v, c.v))):
        assert same_bits(big[which][blocks:], codes[which])
        assert same_bits(got, R.values(*R.quantise(x, 128)).float().to(torch.bfloat16))


def test_slots_past_4_gib():
    """The same of contiguous slots."""
    cap = 5 * 2 ** 20
    c = Call(71, [1, 3], [0, 700], hk=8, share=1)
    big = [torch.empty((2, 8, cap, *x[1].shape[3:]), dtype=x[1].dtype, device="cuda") for x in c.codes + c.params]
    for x, y in zip(big, c.codes + c.params):
        x[:, :, :y[1].shape[2]] = y[1]
    c.attend()
    out, lse = c.out[1].clone(), c.lse[1].clone()
    codes, params = c.cache.stored(c.k, c.v, c.cu, c.lens)
    c.opts.update(cache_k_params=big[2], cache_v_params=big[3])
    c.codes[:2] = [(None, big[0]), (None, big[1])]
    for call in (c.attend, c.write):
        for x, y in zip(big, c.cache.codes + c.cache.params):
            x[:, :, :y.shape[2]] = y.cuda()
        call()
        torch.cuda.synchronize()
        for which in range(2):
            n = codes[which].shape[2]
            assert same_bits(big[which][:, :, :n], codes[which]) and same_bits(big[2 + which][:, :, :n], params[which])
    assert same_bits(c.out[1], out) and same_bits(c.lse[1], lse)
    k, v = torch.empty_like(c.dev[1]), torch.empty_like(c.dev[2])
    binding.prefill_attn_cache4_read(big[0], big[1], c.meta[0], c.offsets, k, v, **c.opts)
    for got, x in ((k, c.k), (v, c.v)):
        assert same_bits(got, R.values(*R.quantise(x, 128)).float().to(torch.bfloat16))


def test_equal_inputs_give_equal_bits():
    outs = []
    for _ in range(3):
        c = Call(9, [1] * 5, [5000, 3, 777, 12000, 64], hk=4, share=2)
        c.attend()
        outs.append((c.out[1].clone(), c.lse[1].clone()))
    for o in outs[1:]:
        assert same_bits(o[0], outs[0][0]) and same_bits(o[1], outs[0][1])


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("new", [[1, 4, 1], [1, 400, 300]])
def test_rotary(block, new):
    """The attention call's rotary embedding: q and the cached key as a call on rotated tensors has them."""
    theta = 10000.0
    c = Call(10, new, [100, 257, 0], hk=1, share=16, group=64, block=block)
    c.attend(rope_theta=theta)
    assert c.expanded == (max(new) > 100)
    rot = [torch.empty_like(x) for x in (c.q, c.k)]
    for b, p in enumerate(c.lens):
        rows = slice(c.cu[b], c.cu[b + 1])
        pos = p + torch.arange(c.new[b])
        for x, y in zip((c.q, c.k), rot):
            y[rows] = R.rotate(x[rows], pos, theta).to(torch.bfloat16)
    e = Call(10, new, [100, 257, 0], hk=1, share=16, group=64, block=block)
    e.q, e.k = rot
    e.dev[:2] = [x.cuda() for x in rot]
    e.attend()
    torch.cuda.synchronize()
    # a rotated value may round the other way (fp32 against 64 bits): one step of bf16 in few places,
    # which moves a score by 2^-8 |q| |k| scale at those; the outputs agree within a bf16 step of the largest
    a, b = c.out[1].double().cpu(), e.out[1].double().cpu()
    assert (a - b).abs().max() <= 8 * R.U * b.abs().max()
    # the call's own write and prefill_attn_cache4_write rotate alike
    w = Call(10, new, [100, 257, 0], hk=1, share=16, group=64, block=block)
    w.write(rope_theta=theta)
    for which in range(2):
        assert same_bits(w.codes[which][1], c.codes[which][1]) and same_bits(w.params[which][1], c.params[which][1])


# ---------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("block", [0, 8, 64])
@pytest.mark.parametrize("d,group", DIMS)
def test_write(d, group, block):
    c = Call(20, [1, 0, 33, 130, 2], [0, 7, 31, 5, 1000], d, hk=3, group=group, block=block)
    c.write()
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == 0
    c.check_cache()
    c.guards()


def edge_rows(d):
    """Rows at the format's edges: constants, one outlier, ties, tiny and huge ranges, signed zeros."""
    x = torch.zeros((12, 1, d))
    x[1] = 3.25
    x[2] = -1e-30
    x[3, 0, 5] = 100.0
    x[4] = torch.arange(d) % 16                               # codes without a rounding
    x[5] = torch.arange(d) % 31 * 0.5                         # ties
    x[6] = 1e-38 * (torch.arange(d) % 7)                      # a scale below the smallest normal number
    x[7] = 2.0 ** -120 * (torch.arange(d) % 3)
    x[8] = 1e38 * ((torch.arange(d) % 3) - 1)
    x[9, 0, ::2] = -0.0
    x[10] = 1000.0 + torch.arange(d) * 4
    x[11, 0, -1] = -7.0
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("d,group", DIMS)
def test_format_edges(d, group):
    c = Call(21, [12], [4], d, hk=1, share=1, group=group)
    c.k = edge_rows(d)
    c.v = edge_rows(d).flip(0)
    c.dev[1], c.dev[2] = c.k.cuda(), c.v.cuda()
    c.write()
    c.check_cache()
    k, v = torch.empty_like(c.dev[1]), torch.empty_like(c.dev[2])
    binding.prefill_attn_cache4_read(c.codes[0][1], c.codes[1][1], c.meta[0], c.offsets, k, v, **c.opts)
    torch.cuda.synchronize()
    for x, got in ((c.k, k), (c.v, v)):
        codes, params = R.quantise(x, group)
        assert same_bits(got, R.values(codes, params).float().to(torch.bfloat16))
        # within half a step, the scale's own rounding over 15 steps, and the value's rounding
        y = x.double().unflatten(-1, (-1, group))
        span = (y.amax(-1) - y.amin(-1))[..., None]
        bound = span / 30 + span * R.U + y.abs() * R.U + 15 * 2.0 ** -126
        assert ((got.cpu().double().unflatten(-1, (-1, group)) - y).abs() <= bound).all()


@pytest.mark.parametrize("block", [0, 8, 64])
@pytest.mark.parametrize("d,group", DIMS)
def test_read(d, group, block):
    g = torch.Generator().manual_seed(22)
    starts, lens = [0, 3, 31, 100, 9], [1, 0, 129, 33, 2]
    cache = R.Cache(g, 5, 160, 3, d, group, block)
    t, cu = sum(lens), cumulative(lens)
    codes, params = [x.cuda() for x in cache.codes], [x.cuda() for x in cache.params]
    out = [guarded(torch.full((t, 3, d), math.nan, dtype=torch.bfloat16)) for _ in range(2)]
    binding.prefill_attn_cache4_read(*codes, i32(cu), i32(starts), out[0][1], out[1][1], cache_k_params=params[0],
                                     cache_v_params=params[1], block_table=None if cache.table is None else cache.table.cuda())
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == 0
    for which in range(2):
        want = torch.empty((t, 3, d), dtype=torch.bfloat16)
        for b in range(5):
            for h in range(3):
                rows = cache.rows(which, b, h, starts[b] + lens[b], starts[b])
                want[cu[b]:cu[b + 1], h] = R.values(*rows).float().to(torch.bfloat16)
        assert same_bits(out[which][1], want)
        assert (out[which][0][:GUARD] == 0x5a).all() and (out[which][0][-GUARD:] == 0x5a).all()


# ---------------------------------------------------------------------------
# metadata, streams, graphs, runs of calls
# ---------------------------------------------------------------------------

def test_bad_sequences_are_skipped():
    """A sequence whose table names a block outside the pool, or whose lengths disagree: nothing of it is touched."""
    c = Call(30, [1, 2, 1], [40, 20, 70], block=16)
    table = c.opts["block_table"]
    table[1, 1] = c.cache.codes[0].shape[0]
    c.attend()
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
    out, lse, bound, _ = R.attention(c.cache, c.q, c.k, c.v, c.cu, c.lens, c.scale)
    got = c.out[1].double().cpu()
    assert got[1:3].isnan().all() and c.lse[1][1:3].isnan().all()
    for rows in (slice(0, 1), slice(3, 4)):
        assert ((got[rows] - out[rows]).abs() <= bound[rows]).all()
    slot, row = c.cache.at(1, torch.arange(20, 22))
    assert same_bits(c.codes[0][1][slot.cuda(), :, row.cuda()], c.cache.codes[0][slot, :, row])
    for call in (c.write, c.attend):
        table[1, 1] = -1
        call()
        assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
    e = Call(31, [1, 1], [40, 20])
    e.meta[1][2] += 1
    e.attend()
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
    assert e.out[1][1].isnan().all() and not e.out[1][0].isnan().any()


def test_bad_chunks_are_skipped():
    c = Call(35, [400, 250, 1], [40, 20, 70], hk=1, share=16, block=16)
    c.opts["block_table"][1, 1] = c.cache.codes[0].shape[0]
    c.attend()
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
    assert c.expanded
    out, _, bound, _ = R.attention(c.cache, c.q, c.k, c.v, c.cu, c.lens, c.scale, tiles=True)
    got = c.out[1].double().cpu()
    assert got[400:650].isnan().all()
    for rows in (slice(0, 400), slice(650, 651)):
        assert ((got[rows] - out[rows]).abs() <= bound[rows]).all()


def test_captured_calls_read_their_metadata_at_replay():
    c = Call(32, [1] * 4, [300, 5, 64, 1000], hk=4, block=16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attend()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.attend()
        want = c.out[1].clone()
        c.out[1].fill_(math.nan)
        for _ in range(3):
            graph.replay()
        side.synchronize()
        assert same_bits(c.out[1], want)
        lens = [17, 900, 0, 33]
        c.cache.spoil([max(a, b) for a, b in zip(lens, c.lens)])
        c.offsets.copy_(i32(lens))
        c.meta[1].copy_(i32(cumulative([p + 1 for p in lens])))
        d = Call(32, [1] * 4, lens, hk=4, block=16, slack=103)  # as many blocks
        for a, b in zip(c.codes + c.params, d.codes + d.params):
            a[1].copy_(b[1])
        graph.replay()
        side.synchronize()
        d.attend()
        side.synchronize()
        assert same_bits(c.out[1], d.out[1]) and same_bits(c.lse[1], d.lse[1])


@pytest.mark.parametrize("new", [[600], [300, 1, 129]])
def test_captured_chunks_read_their_metadata_at_replay(new):
    c = Call(36, new, [300, 5, 64][:len(new)], hk=1, share=24, block=16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.attend()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.attend()
    assert c.expanded
    # other lengths of the same total, and fewer tokens
    for seed, fewer, lens in ((37, new[::-1], [129, 0, 300][:len(new)]), (38, [5, 2, 1][:len(new)], [200, 9, 300][:len(new)]),
                              (39, [400, 0, 1][:len(new)], [37, 300, 5][:len(new)])):
        pad = sum(new) - sum(fewer)
        cap = c.cache.table.shape[1] * 16
        d = Call(seed, fewer, lens, hk=1, share=24, block=16, pad=pad, slack=cap - max(p + n for p, n in zip(lens, fewer)))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for a, b in zip(c.codes + c.params + [c.out, c.lse], d.codes + d.params + [d.out, d.lse]):
                a[1].copy_(b[1])
            for a, b in zip([*c.dev, *c.meta, c.offsets, c.opts["block_table"]],
                            [*d.dev, *d.meta, d.offsets, d.opts["block_table"]]):
                a.copy_(b)
            graph.replay()
        side.synchronize()
        d.codes, d.params, d.out, d.lse = c.codes, c.params, c.out, c.lse
        d.check(tiles=True)


def test_many_paged_sequences():
    """More than a CTA keeps at hand, in blocks; one sequence's table names a block outside the pool."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 90, (400,), generator=g).tolist()
    for bad in (None, 257):
        c = Call(50, [1] * 400, lens, d=64, hk=1, share=2, group=32, block=8)
        if bad is None:
            c.attend()
            c.check()
            continue
        c.opts["block_table"][bad, 0] = -5
        c.attend()
        torch.cuda.synchronize()
        assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
        out, _, bound, _ = R.attention(c.cache, c.q, c.k, c.v, c.cu, c.lens, c.scale)
        got = c.out[1].double().cpu()
        there = torch.arange(400) != bad
        assert got[bad].isnan().all() and ((got - out).abs() <= bound)[there].all()


def test_read_into_tensors_that_are_16_byte_aligned():
    g = torch.Generator().manual_seed(23)
    cache = R.Cache(g, 1, 200, 2, 128, 128)
    codes, params = [x.cuda() for x in cache.codes], [x.cuda() for x in cache.params]
    buf = [torch.full((70 * 256 + 16,), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = buf[0][8:8 + 70 * 256].view(70, 2, 128), buf[1][:70 * 256].view(70, 2, 128)
    assert k.data_ptr() % 32 == 16
    binding.prefill_attn_cache4_read(*codes, i32([0, 70]), i32([100]), k, v, cache_k_params=params[0], cache_v_params=params[1])
    for which, got in enumerate((k, v)):
        for h in range(2):
            assert same_bits(got[:, h], R.values(*cache.rows(which, 0, h, 170, 100)).float().to(torch.bfloat16))
    assert buf[0][:8].isnan().all() and buf[0][-8:].isnan().all() and buf[1][-16:].isnan().all()


def test_threads_on_one_stream():
    """Calls of several host threads at once on one stream run one after the other."""
    calls = [Call(60 + i, new, lens, hk=2, share=16, block=16)
             for i, (new, lens) in enumerate([([1] * 3, [2000, 77, 500]), ([300, 1, 129], [400, 5, 64]), ([600], [100])])]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with concurrent.futures.ThreadPoolExecutor(3) as pool:
        for _ in range(5):
            list(pool.map(lambda c: c.attend(stream=stream), calls))
    stream.synchronize()
    for c in calls:
        c.check(tiles=max(c.new) > 16)


@pytest.mark.parametrize("new", [[1] * 3, [300, 1, 129], [500]])
def test_two_streams_at_once(new):
    calls = [Call(33 + i, new, [2000, 77, 500][:len(new)], hk=2, share=16) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s in zip(calls, streams):
            c.attend(stream=s)
    for c in calls:
        c.check(tiles=max(new) > 16)


@pytest.mark.parametrize("block", [0, 16])
def test_a_conversation(block):
    """A prompt written from elsewhere, decode steps that append to the cache, and the cache read back: each step
    attends what the one before stored."""
    d, group, hk, share = 64, 32, 2, 4
    c = Call(40, [50, 3], [0, 0], d, hk, share, group, block, slack=20)
    c.write()
    codes, params = c.cache.stored(c.k, c.v, c.cu, c.lens)
    lens = [50, 3]
    for step in range(4):
        n = Call(41 + step, [1 + step, 1], lens, d, hk, share, group)
        cache = c.cache
        cache.codes, cache.params = codes, params
        out, lse, bound, lbound = R.attention(cache, n.q, n.k, n.v, n.cu, lens, n.scale)
        o, z = torch.empty_like(n.dev[0]), torch.empty_like(n.lse[1])
        binding.prefill_attn_varlen_cache4(*n.dev, *n.meta, c.codes[0][1], c.codes[1][1], n.offsets, o, z, scale=n.scale,
                                           **c.opts)
        torch.cuda.synchronize()
        assert ((o.double().cpu() - out).abs() <= bound).all() and ((z.double().cpu() - lse).abs() <= lbound).all()
        codes, params = cache.stored(n.k, n.v, n.cu, lens)
        lens = [p + m for p, m in zip(lens, n.new)]
    for which in range(2):
        assert same_bits(c.codes[which][1], codes[which]) and same_bits(c.params[which][1], params[which])
    k, v = (torch.empty((sum(lens), hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    binding.prefill_attn_cache4_read(c.codes[0][1], c.codes[1][1], i32(cumulative(lens)), i32([0, 0]), k, v, **c.opts)
    torch.cuda.synchronize()
    c.cache.codes, c.cache.params = codes, params
    cu = cumulative(lens)
    for which, got in enumerate((k, v)):
        for b in range(2):
            for h in range(hk):
                want = R.values(*c.cache.rows(which, b, h, lens[b])).float().to(torch.bfloat16)
                assert same_bits(got[cu[b]:cu[b + 1], h], want)
