"""GPU tests of the long-context calls: windowed attention with sink tokens, a
prefix that the batch shares, key weights and eviction, each against its plain
64-bit form (tests/long_reference.py, where the tolerances are derived)."""
import math

import pytest
import torch

from prefill_phase_attention_gb300 import binding
from tests import long_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from prefill_phase_attention_gb300 import build
    build.build()
    binding.load()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")


class Call:
    """Inputs of one call on the CPU, their GPU copies, and the outputs in guarded buffers."""

    GUARD = 2048

    def __init__(self, seed, new, lens, d=64, hk=2, group=2, block=0, int8=False, prefix=0, slack=3):
        g = torch.Generator().manual_seed(seed)
        self.new, self.lens, self.hk, self.group, self.d = new, lens, hk, group, d
        cap = max(p + n for p, n in zip(lens, new)) + slack
        self.cache = R.Cache(g, lens, cap, hk, d, block, int8, prefix)
        t = sum(new)
        self.q = torch.randn((t, hk * group, d), generator=g).to(torch.bfloat16)
        self.k = torch.randn((t, hk, d), generator=g).to(torch.bfloat16)
        self.v = torch.randn((t, hk, d), generator=g).to(torch.bfloat16)
        self.cu = R.cumulative(new)
        self.scale = d ** -0.5
        self.weights = torch.rand(self.cache.shape[:-1], generator=g)
        cu_k = R.cumulative([p + n for p, n in zip(lens, new)])
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.meta = (i32(self.cu), i32(cu_k))
        self.offsets = i32(lens)
        self.dev = [x.cuda() for x in (self.q, self.k, self.v)]
        self.data = [self.guarded(x) for x in self.cache.data]
        self.sc = [None if x is None else self.guarded(x) for x in self.cache.scale]
        self.out = self.guarded(torch.full(self.q.shape, math.nan, dtype=torch.bfloat16))
        self.lse = self.guarded(torch.full((t, hk * group), math.nan))
        c = self.cache
        self.opts = dict(block_table=None if c.table is None else c.table.cuda())
        self.scales = dict(cache_k_scale=self.sc[0][1] if self.sc[0] else None,
                           cache_v_scale=self.sc[1][1] if self.sc[1] else None)
        self.pre = {}
        if prefix and block:
            self.pre = dict(prefix_table=c.prefix_table.cuda(), prefix_len=prefix)
        elif prefix:
            up = lambda x: None if x is None else x.cuda()  # noqa: E731
            self.pre = dict(prefix_k=up(c.pre_data[0]), prefix_v=up(c.pre_data[1]), prefix_len=prefix,
                            prefix_k_scale=up(c.pre_scale[0]), prefix_v_scale=up(c.pre_scale[1]))

    def guarded(self, x):
        """(buffer with bands on both sides, the view that holds x)."""
        n = x.numel()
        buf = torch.empty(n + 2 * self.GUARD, dtype=x.dtype, device="cuda")
        R.bits(buf).fill_(0x5a)
        view = buf[self.GUARD:self.GUARD + n].view(x.shape)
        view.copy_(x)
        return buf, view

    def guards(self):
        for buf, _ in self.data + [x for x in self.sc if x] + [self.out, self.lse]:
            b = R.bits(buf)
            assert (b[:self.GUARD] == 0x5a).all() and (b[-self.GUARD:] == 0x5a).all(), "write outside a buffer"

    def tensors(self):
        return (*self.dev, *self.meta, self.data[0][1], self.data[1][1], self.offsets, self.out[1], self.lse[1])

    def sinks(self, window, sinks, theta=0.0, **kw):
        binding.prefill_attn_varlen_sinks(*self.tensors(), window=window, sink_tokens=sinks, scale=self.scale,
                                          rope_theta=theta, **self.opts, **self.scales, **kw)

    def prefix(self, causal=True, theta=0.0, **kw):
        binding.prefill_attn_varlen_prefix(*self.tensors(), scale=self.scale, causal=causal, rope_theta=theta,
                                           **self.opts, **self.scales, **self.pre, **kw)

    def check(self, theta=0.0, skipped=(), **kw):
        """out, lse and the caches against the plain form; sequences in `skipped` were left alone."""
        torch.cuda.synchronize()
        self.guards()
        ref, lse, mag = R.attention(self.cache, self.q, self.k, self.v, self.new, self.scale, theta=theta, **kw)
        got, got_lse = self.out[1].cpu().double(), self.lse[1].cpu().double()
        rows = torch.ones(len(self.q), dtype=torch.bool)
        for b in skipped:
            rows[self.cu[b]:self.cu[b + 1]] = False
        assert got[~rows].isnan().all() and got_lse[~rows].isnan().all(), "rows of a skipped sequence were written"
        # a rotated q or k may differ from the plain rotation by a bf16 rounding: 2^-8 of each product
        score = R.SCORE + (2 * R.BF16 if theta else 0.0)
        tol = R.BF16 * (mag * (2 if self.cache.int8 else 1) + ref.abs()) + score * mag + 1e-6
        err = (got - ref).abs()[rows]
        assert (err <= tol[rows]).all(), f"out off by {err.max():.3e}, {(err / tol[rows]).max():.2f} of the tolerance"
        err = (got_lse - lse).abs()[rows]
        assert (err <= score).all(), f"lse off by {err.max():.3e}"
        if theta:
            return
        for w, new in ((0, self.k), (1, self.v)):
            cu = list(self.cu)
            data, scale = self.cache.written(w, new, cu) if not skipped else (None, None)
            if data is None:
                continue
            assert torch.equal(R.bits(self.data[w][1].cpu()), R.bits(data)), "cache differs"
            if scale is not None:
                assert torch.equal(R.bits(self.sc[w][1].cpu()), R.bits(scale)), "cache scales differ"


def ok():
    assert binding.prefill_attn_device_status() == 0


# --------------------------------------------------------------------------- sink tokens

@pytest.mark.parametrize("block", [0, 16, 128])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,group", [(32, 1), (64, 4), (128, 2)])
def test_sinks_decode_and_chunks(d, group, int8, block):
    """Decode rows, short chunks, an empty sequence and a fresh one; sinks of one token and of several tiles."""
    new, lens = [1, 5, 0, 1, 33, 2], [700, 0, 40, 128, 390, 1]
    for i, (window, sinks) in enumerate([(1, 1), (64, 4), (200, 130), (257, 300), (4000, 7), (2 ** 31 - 1, 2 ** 31 - 1)]):
        c = Call(10 + i, new, lens, d, 2, group, block, int8)
        c.sinks(window, sinks)
        c.check(window=window, sinks=sinks)
    ok()


@pytest.mark.parametrize("schedule", [0, 1, 2, 3])
@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("d,group", [(64, 1), (128, 8)])
def test_sinks_prompts(d, group, block, schedule):
    """Prompts longer than the window: tiles between the sinks and the window are skipped."""
    c = Call(30, [900, 131, 1], [0, 517, 64], d, 1, group, block)
    c.sinks(150, 5, schedule=schedule)
    c.check(window=150, sinks=5)
    ok()


@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 128), (127, 129), (128, 128), (129, 256), (300, 257), (257, 500), (640, 5)])
@pytest.mark.parametrize("block,int8", [(0, False), (16, False), (0, True), (16, True)])
def test_sinks_of_several_tiles_under_prompts(block, int8, window, sinks):
    """Units of two query tiles on every side of where the window leaves the sink tiles."""
    for group, lens in ((1, [0, 77, 640]), (4, [128, 0, 333])):
        c = Call(31, [1030, 257, 700], lens, 64, 1, group, block, int8)
        c.sinks(window, sinks, schedule=2)
        c.check(window=window, sinks=sinks)
    ok()


@pytest.mark.parametrize("window,sinks", [(2500, 4), (6000, 200), (100, 129)])
@pytest.mark.parametrize("block,int8", [(0, False), (16, False), (0, True)])
def test_sinks_one_long_row_is_split(block, int8, window, sinks):
    """One decode row over many tiles: its keys are split between CTAs and joined."""
    c = Call(40, [1], [4099], 128, 2, 4, block, int8)
    c.sinks(window, sinks)
    # (a window of at most 8 tiles is not: it runs without the merge; neither needs a scheduler of its own)
    assert binding.prefill_attn_last_launch_count() == (2 if (window + sinks) // 128 + 3 > 8 else 1)
    c.check(window=window, sinks=sinks)
    ok()


def test_sinks_zero_is_the_plain_window():
    c = Call(50, [1, 70], [300, 200], 64, 2, 2)
    c.sinks(90, 0)
    c.check(window=90)
    ok()


@pytest.mark.parametrize("block", [0, 32])
def test_sinks_rotary(block):
    c = Call(51, [3, 40], [300, 0], 64, 2, 2, block)
    c.sinks(90, 4, theta=1e4)
    c.check(theta=1e4, window=90, sinks=4)
    ok()


# --------------------------------------------------------------------------- shared prefix

@pytest.mark.parametrize("block", [0, 16, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,group", [(32, 4), (64, 1), (128, 8)])
def test_prefix_of_every_length(d, group, int8, block):
    """Prefixes that end inside, at and past a tile; decode rows, chunks, empty and fresh sequences."""
    new, lens = [1, 4, 0, 1, 20, 1], [0, 130, 9, 300, 0, 128]
    for i, prefix in enumerate([1, 127, 128, 129, 700]):
        c = Call(60 + i, new, lens, d, 2, group, block, int8, prefix)
        c.prefix()
        c.check()
    ok()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("schedule", [0, 1, 2, 3])
def test_prefix_with_prompts(causal, schedule):
    c = Call(70, [300, 1, 129], [0, 70, 5], 128, 2, 2, prefix=389)
    c.prefix(causal=causal, schedule=schedule)
    c.check(causal=causal)
    ok()


@pytest.mark.parametrize("block", [0, 16])
def test_prefix_split_between_many_blocks(block):
    """A long prefix under a few rows: pieces, and a long own context cut into pieces as well."""
    c = Call(71, [1, 1, 2], [3000, 1, 0], 128, 1, 4, block, prefix=6001)
    c.prefix()
    c.check()
    ok()


def test_prefix_of_nothing_is_the_plain_call():
    c = Call(72, [1, 30], [200, 0], 64, 2, 2)
    one = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    c.pre = dict(prefix_k=one, prefix_v=one.clone(), prefix_len=0)
    c.prefix()
    c.check()
    ok()


@pytest.mark.parametrize("block", [0, 32])
def test_prefix_rotary_counts_from_the_prefix(block):
    c = Call(73, [2, 17], [100, 0], 64, 2, 2, block, prefix=150)
    c.prefix(theta=1e4)
    c.check(theta=1e4)
    ok()


def test_prefix_bad_block_rejects_the_call():
    c = Call(74, [1, 3], [20, 0], 64, 2, 2, 16, prefix=40)
    c.pre["prefix_table"][1] = 10 ** 6
    before = [x[1].clone() for x in c.data]
    c.prefix()
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() & binding.DEVERR_METADATA
    assert c.out[1].isnan().all() and c.lse[1].isnan().all()
    assert all(torch.equal(R.bits(a), R.bits(b[1])) for a, b in zip(before, c.data))


@pytest.mark.parametrize("call", ["sinks", "prefix"])
def test_inconsistent_sequence_is_skipped(call):
    c = Call(75, [1, 3, 2], [20, 7, 200], 64, 2, 2, prefix=40 if call == "prefix" else 0)
    c.offsets[1] = 8  # disagrees with cu_seqlens_k
    before = [x[1][1].clone() for x in c.data]
    if call == "sinks":
        c.sinks(64, 4)
        c.check(skipped=[1], window=64, sinks=4)
    else:
        c.prefix()
        c.check(skipped=[1])
    assert binding.prefill_attn_device_status() & binding.DEVERR_METADATA
    assert all(torch.equal(R.bits(a), R.bits(b[1][1])) for a, b in zip(before, c.data))


# --------------------------------------------------------------------------- key weights

def weigh(c, lse=None, causal=True, window=0, sinks=0, theta=0.0, **kw):
    """Runs the call on c's weights and compares every row of them."""
    if lse is None:
        lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale, causal, window, sinks, theta)[1].float()
    buf, w = c.guarded(c.weights)
    binding.prefill_attn_key_weights(c.dev[0], c.dev[1], *c.meta, c.data[0][1], c.offsets, lse.cuda(), w, scale=c.scale,
                                     causal=causal, window=window, sink_tokens=sinks, rope_theta=theta,
                                     prefix_len=c.cache.prefix, cache_k_scale=c.scales["cache_k_scale"], **c.opts, **kw)
    torch.cuda.synchronize()
    b = R.bits(buf)
    assert (b[:c.GUARD] == 0x5a).all() and (b[-c.GUARD:] == 0x5a).all(), "write outside weights"
    ref = R.key_weights(c.cache, c.q, c.k, c.new, lse, c.scale, c.weights, causal, window, sinks, theta)
    got = w.cpu().double()
    same = ref == c.weights.double()  # rows no key of this call has: untouched, bit for bit
    assert torch.equal(got[same], ref[same])
    # 2^-11 of a term for its score; n fp32 additions of terms of one sign: n 2^-24 of the sum
    tol = (R.SCORE + (2 * R.BF16 if theta else 0.0) + max(c.new) * c.group * 2.0 ** -24) * ref.abs() + 1e-6
    err = (got - ref).abs()
    assert (err <= tol).all(), f"weights off by {err.max():.3e}, {(err / tol).max():.2f} of the tolerance"
    return w


@pytest.mark.parametrize("block", [0, 16, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d,group", [(32, 4), (64, 1), (128, 8)])
def test_key_weights(d, group, int8, block):
    c = Call(80, [1, 5, 0, 1, 150, 2], [700, 0, 40, 128, 390, 1], d, 2, group, block, int8)
    weigh(c)
    weigh(c, window=100, sinks=3)
    weigh(c, window=2 ** 31 - 1, sinks=2 ** 31 - 1)
    ok()


@pytest.mark.parametrize("group,causal", [(1, True), (3, True), (4, False), (128, True)])
def test_key_weights_of_prompts(group, causal):
    new = [513, 128, 1, 200] if group < 128 else [9, 1]
    lens = [0, 129, 0, 5] if group < 128 else [0, 140]
    c = Call(81, new, lens, 128, 1, group)
    weigh(c, causal=causal)
    ok()


def test_key_weights_are_probabilities():
    """The weights that a fresh prompt's keys collect sum to its number of queries times heads."""
    c = Call(82, [333], [0], 64, 2, 2)
    w = weigh(c)
    total = w[0, :, :333].double().sum(-1).cpu()
    assert (total - 333 * 2).abs().max() <= 333 * 2 * R.SCORE


def test_key_weights_rotary_and_prefix():
    c = Call(83, [3, 40], [120, 0], 64, 2, 2, prefix=77)
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale, theta=1e4)[1].float()
    weigh(c, lse, theta=1e4)
    ok()


def test_key_weights_twice_gives_equal_bits():
    c = Call(84, [200, 1], [100, 900], 128, 2, 4)
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale)[1].float()
    assert torch.equal(weigh(c, lse), weigh(c, lse))


# --------------------------------------------------------------------------- eviction

def evict(c, weights, budget, sinks, recent, lens=None, index=True, kept="new", bad=()):
    lens = c.lens if lens is None else lens
    dev = torch.tensor(lens, dtype=torch.int32).cuda()
    new = torch.full_like(dev, -7)
    buf, w = c.guarded(weights)
    kw = w if kept == "same" else torch.full_like(w, 9.0) if kept == "new" else None
    idx = torch.full((len(lens), c.hk, budget), -9, dtype=torch.int32, device="cuda") if index else None
    binding.prefill_attn_evict(c.data[0][1], c.data[1][1], w, dev, new, idx, kw, budget=budget, sink_tokens=sinks,
                               recent_tokens=recent, **c.opts, **c.scales)
    torch.cuda.synchronize()
    c.guards()
    want = [[x.clone() for x in c.cache.data], [None if x is None else x.clone() for x in c.cache.scale]]
    want_w = weights.clone() if kept == "same" else torch.full_like(weights, 9.0)
    for b, n in enumerate(lens):
        if b in bad:
            assert new[b] == -7 and (idx is None or (idx[b] == -9).all())
            continue
        m = min(n, budget)
        assert int(new[b]) == m
        for h in range(c.hk):
            slot, row = c.cache.at(b, torch.arange(n))
            keep = R.evicted(weights[slot, h, row], budget, sinks, recent)
            if idx is not None:
                assert torch.equal(idx[b, h, :m].cpu().long(), keep), f"sequence {b}, head {h}"
                assert (idx[b, h, m:] == -1).all()
            want_w[slot[:m], h, row[:m]] = weights[slot[keep], h, row[keep]]
            for w_ in range(2):
                want[0][w_][slot[:m], h, row[:m]] = c.cache.data[w_][slot[keep], h, row[keep]]
                if c.cache.int8:
                    want[1][w_][slot[:m], h, row[:m]] = c.cache.scale[w_][slot[keep], h, row[keep]]
    for w_ in range(2):
        assert torch.equal(R.bits(c.data[w_][1].cpu()), R.bits(want[0][w_])), "cache differs"
        if c.cache.int8:
            assert torch.equal(R.bits(c.sc[w_][1].cpu()), R.bits(want[1][w_])), "scales differ"
    if kw is not None:
        assert torch.equal(R.bits(kw.cpu()), R.bits(want_w)), "kept weights differ"
    if kept != "same":
        assert torch.equal(R.bits(w.cpu()), R.bits(weights)), "weights were changed"


def weights_for(c, seed, kind):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(c.cache.shape[:-1], generator=g)
    if kind == "ties":
        w = (w * 4).floor() / 4
    if kind == "special":
        for x in (math.nan, math.inf, -math.inf, 0.0, -0.0, -1.5, 1e-42):
            w[torch.rand(w.shape, generator=g) < 0.08] = x
    return w


@pytest.mark.parametrize("block", [0, 8, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_evict(d, int8, block):
    """Every length class: empty, one token, below, at and just above the budget, far above it."""
    lens = [0, 1, 90, 100, 101, 733, 2100]
    for i, (kind, sinks, recent) in enumerate([("plain", 4, 16), ("ties", 0, 0), ("special", 3, 97), ("special", 1, 5)]):
        c = Call(90 + i, [0] * len(lens), lens, d, 3, 1, block, int8)
        evict(c, weights_for(c, i, kind), 100, sinks, recent, kept=["new", "same", "new", "none"][i], index=i != 1)
    ok()


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (2049, 4, 1000), (4999, 0, 3)])
@pytest.mark.parametrize("kept", ["new", "same"])
def test_evict_extremes(budget, sinks, recent, kept):
    """Lengths on both sides of what one CTA selects alone (4096 tokens)."""
    c = Call(95, [0] * 4, [5000, 3000, 4096, 4097], 64, 2, 1)
    evict(c, weights_for(c, 1, "ties"), budget, sinks, recent, kept=kept)
    ok()


@pytest.mark.parametrize("int8,block", [(False, 0), (True, 0), (False, 16)])
def test_evict_long_sequences(int8, block):
    """Shares of a cluster's CTAs past what their threads hold in registers."""
    c = Call(94, [0, 0], [40001, 16500], 32, 1, 1, block, int8)
    evict(c, weights_for(c, 3, "special"), 9001, 4, 100, kept="same")
    ok()


@pytest.mark.parametrize("heads", [1, 200])
@pytest.mark.parametrize("spread", [1, 7, 10, 14, 18, 25])
def test_evict_weights_that_share_leading_bits(spread, heads):
    """Weights within 2^spread steps of fp32 of one another: the choice is made after every possible number of
    digits, and with more and fewer equal weights than are compared at once; one launch, and two."""
    c = Call(93, [0] * 6, [129, 133, 700, 2049, 5000, 9000] if heads == 1 else [129, 133, 135, 300, 700, 1200], 32, heads, 1)
    g = torch.Generator().manual_seed(spread)
    steps = torch.randint(0, 2 ** spread, c.cache.shape[:-1], generator=g, dtype=torch.int32)
    evict(c, (steps + 0x3f800000).view(torch.float32), 128, 3, 20)
    ok()


@pytest.mark.parametrize("lens,block,kept", [([9000, 4097], 0, "same"), ([8193, 300], 16, "new"), ([33500, 4096], 0, "same")])
def test_evict_of_many_long_heads(lens, block, kept):
    """Two launches, the select by clusters: shares that a CTA's threads hold at once, and longer ones."""
    c = Call(92, [0, 0], lens, 32, 77, 1, block)
    evict(c, weights_for(c, 4, "ties" if block else "special"), 1000, 4, 100, kept=kept)
    assert binding.prefill_attn_last_launch_count() == 2
    ok()


def test_evict_equal_weights_keeps_the_first():
    c = Call(96, [0], [1500], 64, 1, 1)
    evict(c, torch.zeros(c.cache.shape[:-1]), 600, 2, 10)
    ok()


def test_evict_skips_a_bad_length_and_a_bad_block():
    c = Call(97, [0] * 3, [200, 300, 250], 64, 2, 1, 16)
    c.opts["block_table"][1, 3] = -1
    evict(c, weights_for(c, 2, "plain"), 100, 2, 10, bad=(1,))
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
    c = Call(98, [0] * 3, [200, 300, 250], 64, 2, 1)
    evict(c, weights_for(c, 2, "plain"), 100, 2, 10, lens=[200, 10 ** 6, 250], bad=(1,))
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA
    evict(Call(98, [0] * 3, [200, 300, 250], 64, 2, 1), weights_for(c, 2, "plain"), 100, 2, 10, lens=[200, -4, 250],
          bad=(1,))
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA


# --------------------------------------------------------------------------- together

@pytest.mark.parametrize("block", [0, 16])
def test_prefill_weigh_evict_decode(block):
    """A prompt is prefilled, its keys weighed, the cache cut back, and a token decoded over what is left."""
    d, hk, group, n, budget = 64, 2, 4, 300, 120
    c = Call(100, [n, n - 61], [0, 0], d, hk, group, block)
    binding.prefill_attn_varlen_ex(*c.tensors(), scale=c.scale, **c.opts)
    c.check()
    lse = c.lse[1].cpu()
    w = weigh(c, lse)
    before = w.cpu()
    lens = torch.tensor(c.new, dtype=torch.int32).cuda()
    kept, index = torch.empty_like(lens), torch.empty((2, hk, budget), dtype=torch.int32, device="cuda")
    binding.prefill_attn_evict(c.data[0][1], c.data[1][1], w, lens, kept, index, w, budget=budget, sink_tokens=4,
                               recent_tokens=32, **c.opts)
    assert kept.tolist() == [budget, budget]
    # the token that follows sees the kept keys and itself
    g = torch.Generator().manual_seed(5)
    q1 = torch.randn((2, hk * group, d), generator=g).to(torch.bfloat16)
    k1, v1 = (torch.randn((2, hk, d), generator=g).to(torch.bfloat16) for _ in range(2))
    out, cu = torch.empty_like(q1).cuda(), torch.tensor([0, 1, 2], dtype=torch.int32).cuda()
    cu_k = torch.tensor([0, budget + 1, 2 * budget + 2], dtype=torch.int32).cuda()
    binding.prefill_attn_varlen_ex(q1.cuda(), k1.cuda(), v1.cuda(), cu, cu_k, c.data[0][1], c.data[1][1], kept, out,
                                   scale=c.scale, **c.opts)
    got = out.cpu().double()
    for b in range(2):
        t = slice(c.cu[b], c.cu[b + 1])
        for h in range(hk * group):
            keep = index[b, h // group].cpu().long()
            slot, row = c.cache.at(b, torch.arange(c.new[b]))
            assert torch.equal(keep, R.evicted(before[slot, h // group, row], budget, 4, 32))
            keys = torch.cat([c.k[t][keep, h // group], k1[b:b + 1, h // group]]).double()
            vals = torch.cat([c.v[t][keep, h // group], v1[b:b + 1, h // group]]).double()
            p = torch.softmax(keys @ q1[b, h].double() * c.scale, 0)
            ref, mag = p @ vals, p @ vals.abs()
            tol = R.BF16 * (mag + ref.abs()) + R.SCORE * mag + 1e-6
            assert ((got[b, h] - ref).abs() <= tol).all()
    ok()


def test_sinks_blocks_between_sinks_and_window_may_be_gone():
    """A streaming server gives back the blocks that no query sees: their table entries may hold anything."""
    c = Call(52, [1, 3], [1000, 700], 64, 2, 2, 16)
    # window 100 over 1000: tiles from position 896 on; over 700 (oldest query at 700): from 512 on
    c.opts["block_table"][0, 8:56] = -1
    c.opts["block_table"][1, 8:32] = 10 ** 6
    c.sinks(100, 4)
    c.check(window=100, sinks=4)
    ok()
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale, window=100, sinks=4)[1].float()
    weigh(c, lse, window=100, sinks=4)
    ok()


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("seqs", [256, 257, 1300])
def test_many_sequences(seqs, block):
    """Both sides of the batch size up to which a few sequences are ranked directly (256, the prefix counted)."""
    new = [(i * 7) % 3 for i in range(seqs)]
    lens = [(i * 37) % 150 for i in range(seqs)]
    c = Call(110, new, lens, 32, 1, 2, block)
    c.sinks(40, 3)
    c.check(window=40, sinks=3)
    weigh(c)
    c = Call(111, new, lens, 32, 1, 2, block, prefix=70)
    c.prefix()
    c.check()
    ok()


def test_many_sequences_with_a_bad_block():
    c = Call(112, [1] * 300, [(i * 11) % 60 for i in range(300)], 32, 1, 1, 16)
    c.opts["block_table"][299, 0] = -1
    c.sinks(40, 3)
    c.check(skipped=[299], window=40, sinks=3)
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA


@pytest.mark.parametrize("block,int8", [(0, False), (0, True), (32, False), (32, True)])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_key_weights_of_mixed_queries(d, block, int8):
    """Sequences of one query row to several Q tiles of them (16, 17 and 32 tokens of 4 heads: 64, 68 and 128 rows),
    many of each, so that a CTA takes units of both kinds in turn."""
    new = [1, 17, 16, 200, 1, 32, 33, 3] * 12
    lens = [(i * 131) % 700 for i in range(len(new))]
    c = Call(120, new, lens, d, 2, 4, block, int8)
    weigh(c)
    ok()


@pytest.mark.parametrize("group", [3, 5, 7, 48])
def test_key_weights_of_groups_that_do_not_divide_a_tile(group):
    """126, 125, 126 and 96 rows in a Q tile; the queries' tails are cut at other places than tokens of 128 rows."""
    c = Call(121, [300, 64, 1], [5, 200, 90], 64, 1, group)
    weigh(c)
    ok()


@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("group", [3, 7, 48, 128])
def test_attention_groups_that_do_not_divide_a_tile(group, block):
    """Query blocks of 42, 18, 2 tokens and of one, whole and in pieces (the merge numbers tokens by block)."""
    new, lens = [45, 1, 4], [5, 1500, 90]
    c = Call(123, new, lens, 64, 1, group, block)
    c.sinks(1200, 4)
    c.check(window=1200, sinks=4)
    c = Call(124, new, lens, 64, 1, group, block, prefix=777)
    c.prefix()
    c.check()
    ok()


@pytest.mark.parametrize("call", ["sinks", "prefix", "weights"])
@pytest.mark.parametrize("new,lens", [([1, 3], [900, 40]), ([1] * 70, list(range(70)))])
def test_rows_behind_the_last_sequence_stay(call, new, lens):
    """A batch padded to a larger total_q: the rows behind are left as they were, and reach no result."""
    c = Call(125, new, lens, 64, 2, 2, prefix=300 if call == "prefix" else 0)
    t, more = sum(new), 140
    big = [torch.cat([x, torch.full((more, *x.shape[1:]), 3.0, dtype=x.dtype, device="cuda")]) for x in c.dev]
    out = torch.full_like(big[0], math.nan)
    lse = torch.full(big[0].shape[:2], math.nan, device="cuda")
    c.dev, c.out, c.lse = big, (c.out[0], out), (c.lse[0], lse)
    if call == "weights":
        w = weigh_padded(c, t)
        assert torch.equal(w, weigh_padded(c, t))
        return
    c.sinks(64, 4) if call == "sinks" else c.prefix()
    torch.cuda.synchronize()
    assert out[t:].isnan().all() and lse[t:].isnan().all()
    c.out, c.lse = (c.out[0], out[:t]), (c.lse[0], lse[:t])
    c.check(**(dict(window=64, sinks=4) if call == "sinks" else {}))
    ok()


def weigh_padded(c, t):
    """Key weights of a padded batch whose first t rows are the sequences'."""
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale)[1].float()
    w = c.weights.cuda()
    padded = torch.cat([lse, torch.full((len(c.dev[0]) - t, lse.shape[1]), -5.0)]).cuda()
    binding.prefill_attn_key_weights(c.dev[0], c.dev[1], *c.meta, c.data[0][1], c.offsets, padded, w, scale=c.scale)
    ref = R.key_weights(c.cache, c.q, c.k, c.new, lse, c.scale, c.weights)
    tol = (R.SCORE + max(c.new) * c.group * 2.0 ** -24) * ref.abs() + 1e-6
    assert ((w.cpu().double() - ref).abs() <= tol).all()
    ok()
    return w


def test_key_weights_under_a_window_of_millions_of_tokens():
    """A window times the heads of a group passes 32 bits; it sees the few tokens of these sequences all the same."""
    c = Call(126, [1, 2, 1], [300, 10, 0], 32, 1, 128)
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale)[1].float().cuda()
    cap, used = (1 << 24) + 64, c.weights.shape[-1]
    keys = torch.zeros((3, 1, cap, 32), dtype=torch.bfloat16, device="cuda")
    keys[:, :, :used] = c.data[0][1]
    got = {}
    for window in (0, 1 << 24):
        w = torch.zeros((3, 1, cap), device="cuda")
        binding.prefill_attn_key_weights(c.dev[0], c.dev[1], *c.meta, keys, c.offsets, lse, w, scale=c.scale, window=window)
        got[window] = w
    assert torch.equal(got[0], got[1 << 24])
    ref = R.key_weights(c.cache, c.q, c.k, c.new, lse.cpu(), c.scale, torch.zeros_like(c.weights))
    tol = (R.SCORE + 2 * 128 * 2.0 ** -24) * ref.abs() + 1e-6
    assert ((got[0][:, :, :used].cpu().double() - ref).abs() <= tol).all()
    ok()


def test_prefix_with_more_units_than_ctas():
    """Whole rounds of prefix units stay uncut, the last round is cut into pieces."""
    c = Call(122, [300, 1, 601], [0, 70, 5], 32, 64, 1, prefix=1111)
    c.prefix()
    c.check()
    ok()


# --------------------------------------------------------------------------- streams, graphs, large caches

def run_all(c, d, st=None):
    """Every long-context call once, on stream st, on the tensors in d; returns what they wrote."""
    kw = dict(scale=c.scale, stream=st, **c.opts)
    args = (d["q"], d["k"], d["v"], *c.meta, d["ck"], d["cv"], c.offsets)
    binding.prefill_attn_varlen_sinks(*args, d["out"], d["lse"], window=90, sink_tokens=4, **kw)
    binding.prefill_attn_varlen_prefix(*args, d["out2"], d["lse2"], **c.pre, **kw)
    binding.prefill_attn_key_weights(d["q"], d["k"], *c.meta, d["ck"], c.offsets, d["lse"], d["w"], window=90, sink_tokens=4, **kw)
    binding.prefill_attn_evict(d["ck"], d["cv"], d["w"], c.offsets, d["kept"], d["index"], d["kw"], budget=60, sink_tokens=4,
                               recent_tokens=8, stream=st, **c.opts)


def tensors(c):
    d = dict(zip("qkv", (x.clone() for x in c.dev)))
    d.update(ck=c.cache.data[0].cuda(), cv=c.cache.data[1].cuda(), w=c.weights.cuda(), kw=c.weights.cuda() * 0)
    d.update(out=torch.zeros_like(d["q"]), out2=torch.zeros_like(d["q"]), kept=torch.zeros_like(c.offsets))
    d.update(lse=torch.zeros(d["q"].shape[:2], device="cuda"), lse2=torch.zeros(d["q"].shape[:2], device="cuda"))
    d.update(index=torch.zeros((len(c.lens), c.hk, 60), dtype=torch.int32, device="cuda"))
    return d


def same(a, b):
    for name in a:
        assert torch.equal(R.bits(a[name]), R.bits(b[name])), name


@pytest.mark.parametrize("block", [0, 16])
def test_graph_replay_gives_the_bits_of_an_eager_call(block):
    """The calls captured once and replayed on other data, between eager calls that outgrow the workspace."""
    st = torch.cuda.Stream()
    mk = lambda seed: Call(seed, [1, 40, 0, 3], [300, 10, 5, 128], 64, 2, 2, block, prefix=200)  # noqa: E731
    c, other = mk(130), mk(131)
    held, start = tensors(c), tensors(c)
    with torch.cuda.stream(st):
        run_all(c, tensors(c), st)  # sizes the workspace
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        run_all(c, held, st)
    want = tensors(c)
    run_all(c, want)  # eager, on the default stream's own workspace
    for _ in range(2):
        for name in start:
            held[name].copy_(start[name])
        g.replay()
        torch.cuda.synchronize()
        same(held, want)
        # larger calls on the graph's stream: its workspace is outgrown, not freed
        big = Call(132, [1] * 90, [200 + i for i in range(90)], 64, 2, 2, block, prefix=900)
        with torch.cuda.stream(st):
            big.sinks(100, 4, stream=st)
            big.prefix(stream=st)
        st.synchronize()
        big.check()
    if not block:  # other data in the captured buffers (a paged call's table would be another)
        for k, t in c.pre.items():
            if torch.is_tensor(t):
                t.copy_(other.pre[k])
        want = tensors(other)
        for name, t in tensors(other).items():
            held[name].copy_(t)
        run_all(c, want)
        g.replay()
        torch.cuda.synchronize()
        same(held, want)
    with torch.cuda.stream(st):
        assert binding.prefill_attn_device_status(st) == 0
    ok()


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
@pytest.mark.parametrize("call", ["sinks", "prefix", "weights"])
def test_capture_on_a_fresh_stream_is_refused(call):
    c = Call(133, [1, 40], [300, 10], 64, 2, 2, prefix=100 if call == "prefix" else 0)
    d = tensors(c)
    st = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with pytest.raises(binding.PrefillAttnError) as err:
        with torch.cuda.graph(g, stream=st):
            if call == "weights":
                binding.prefill_attn_key_weights(d["q"], d["k"], *c.meta, d["ck"], c.offsets, d["lse"], d["w"], stream=st)
            else:
                getattr(c, call)(*((64, 4) if call == "sinks" else ()), stream=st)
    assert err.value.status == 2 and "graph capture" in str(err.value)
    if call != "weights":
        getattr(c, call)(*((64, 4) if call == "sinks" else ()), stream=st)
        torch.cuda.synchronize()
        c.check(**(dict(window=64, sinks=4) if call == "sinks" else {}))


def test_two_streams_at_once():
    """Calls on two streams have workspaces of their own."""
    cs = [Call(134 + i, [1, 50], [2000, 30], 128, 2, 4, prefix=300) for i in range(2)]
    wants = [tensors(c) for c in cs]
    for c, w in zip(cs, wants):
        run_all(c, w)
    torch.cuda.synchronize()
    got, sts = [tensors(c) for c in cs], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for c, d, st in zip(cs, got, sts):
        with torch.cuda.stream(st):
            run_all(c, d, st)
    torch.cuda.synchronize()
    for d, w in zip(got, wants):
        same(d, w)


def large_caches(c):
    """c's caches inside ones of more than 2^32 bytes, in use at the far end: (K, V, place, back); place(t, x) copies
    x to where a tensor of the large caches' rows has it, back(t) is that part of t."""
    hk, d = c.hk, c.d
    if c.cache.block:
        first = 8400  # blocks ahead of the ones in use
        shape = (first + c.cache.shape[0], hk, c.cache.block, d)
        c.opts["block_table"] = c.opts["block_table"] + first
        back = lambda t: t[first:]  # noqa: E731
    else:
        shape, cap = (2, hk, 1_100_000, d), c.cache.shape[2]
        back = lambda t: t[:, :, :cap]  # noqa: E731
    assert math.prod(shape) * 2 > 2 ** 32
    place = lambda t, x: back(t).copy_(x)  # noqa: E731
    big = [torch.empty(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for t, x in zip(big, c.cache.data):
        place(t, x.cuda())
    return *big, place, back


@pytest.mark.parametrize("block,prefix", [(0, 0), (256, 0), (0, 150)])
def test_caches_past_four_gigabytes(block, prefix):
    """The last slot (or the last blocks) of a cache lies more than 2^32 bytes from its start."""
    new, lens = [3, 1], [700, 300]
    c = Call(140, new, lens, 128, 8, 2, block, prefix=prefix)
    ck, cv, place, back = large_caches(c)
    args = (*c.dev, *c.meta, ck, cv, c.offsets, c.out[1], c.lse[1])
    if prefix:
        binding.prefill_attn_varlen_prefix(*args, scale=c.scale, **c.opts, **c.pre)
    else:
        binding.prefill_attn_varlen_sinks(*args, window=90, sink_tokens=4, scale=c.scale, **c.opts)
    for own, big in zip(c.data, (ck, cv)):
        own[1].copy_(back(big))
    c.check(**({} if prefix else dict(window=90, sinks=4)))
    if prefix:
        return
    weights = torch.zeros(ck.shape[:-1], device="cuda")
    place(weights, c.weights.cuda())
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale)[1].float()
    binding.prefill_attn_key_weights(c.dev[0], c.dev[1], *c.meta, ck, c.offsets, lse.cuda(), weights, scale=c.scale, **c.opts)
    ref = R.key_weights(c.cache, c.q, c.k, c.new, lse, c.scale, c.weights)
    assert ((back(weights).cpu().double() - ref).abs() <= R.SCORE * 2 * ref.abs() + 1e-6).all()
    kept, index = torch.zeros_like(c.offsets), torch.zeros((2, c.hk, 200), dtype=torch.int32, device="cuda")
    now = back(weights).cpu()
    binding.prefill_attn_evict(ck, cv, weights, c.offsets, kept, index, weights, budget=200, sink_tokens=4,
                               recent_tokens=16, **c.opts)
    moved = back(cv).cpu()
    for b, n in enumerate(lens):
        slot, row = c.cache.at(b, torch.arange(n))
        for h in (0, c.hk - 1):
            keep = R.evicted(now[slot, h, row], 200, 4, 16)
            assert torch.equal(index[b, h].cpu().long(), keep)
            assert torch.equal(R.bits(moved[slot[:200], h, row[:200]]), R.bits(c.cache.data[1][slot[keep], h, row[keep]]))
    ok()


@pytest.mark.parametrize("call", ["sinks", "prefix"])
def test_without_lse(call):
    """lse is optional, whether units write out themselves or a merge does."""
    c = Call(150, [1, 40], [2000, 10], 64, 2, 2, prefix=300 if call == "prefix" else 0)
    args = c.tensors()[:-1]
    if call == "sinks":
        binding.prefill_attn_varlen_sinks(*args, window=1500, sink_tokens=4, scale=c.scale)
    else:
        binding.prefill_attn_varlen_prefix(*args, scale=c.scale, **c.pre)
    torch.cuda.synchronize()
    kw = dict(window=1500, sinks=4) if call == "sinks" else {}
    ref, lse, _ = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale, **kw)
    assert c.lse[1].isnan().all()
    c.lse[1].copy_(lse)
    c.check(**kw)
    ok()


@pytest.mark.parametrize("seqs", [9, 10, 18, 19, 63, 64])
def test_planned_by_the_kernel_or_by_the_scheduler(seqs):
    """Both sides of the sizes up to which the attention kernel plans for itself (a unit per SM at most, 63 sequences)."""
    hk = 8 if seqs < 40 else 1
    lens = [(i * 977) % 2500 for i in range(seqs)]
    c = Call(160, [1] * seqs, lens, 64, hk, 4, prefix=1500)
    c.prefix()
    c.check()
    c = Call(161, [1 + i % 3 for i in range(seqs)], lens, 64, hk, 4, 32)
    c.sinks(1200, 4)
    c.check(window=1200, sinks=4)
    ok()
