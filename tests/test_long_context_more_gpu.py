"""More GPU tests of the long-context calls: sizes, options and argument shapes at their edges."""
import math

import pytest
import torch

from prefill_phase_attention_gb300 import binding
from tests import long_reference as R
from tests.test_long_context_gpu import Call, evict, ok, weights_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from prefill_phase_attention_gb300 import build
    build.build()
    binding.load()


@pytest.mark.parametrize("seqs,kept", [(64, "new"), (64, "same"), (2, "none")])
def test_evict_with_a_budget_past_the_cache_keeps_everything(seqs, kept):
    """No index is wanted: none of budget entries is made room for (64 sequences of 2^31 - 1 would be 1 TiB)."""
    c = Call(300, [0] * seqs, [(i * 37) % 90 for i in range(seqs)], 64, 2, 1)
    evict(c, weights_for(c, 1, "special"), 2 ** 31 - 1, 2 ** 30, 2 ** 30 - 1, index=False, kept=kept)
    ok()


def test_evict_with_a_budget_past_the_cache_fills_the_index():
    c = Call(301, [0] * 3, [90, 0, 17], 64, 2, 1)
    evict(c, weights_for(c, 1, "plain"), 1000, 600, 300)
    ok()


def swapped(t, a=-1, b=-2):
    """A contiguous tensor of as many elements, two dimensions swapped."""
    return torch.zeros_like(t.transpose(a, b).contiguous())


@pytest.mark.parametrize("name", ["v", "cache_v", "out", "lse", "cache_k_scale", "cache_v_scale"])
@pytest.mark.parametrize("call", ["sinks", "prefix"])
def test_attention_refuses_other_shapes_of_as_many_elements(call, name):
    c = Call(310, [3, 5], [20, 7], 64, 2, 2, int8="scale" in name, prefix=40 if call == "prefix" else 0)
    names = ("q", "k", "v", "cu_seqlens_q", "cu_seqlens_k", "cache_k", "cache_v", "cache_offsets", "out", "lse")
    t = {**dict(zip(names, c.tensors())), **c.scales}
    t[name] = swapped(t[name])
    kw = dict(window=9, sink_tokens=2) if call == "sinks" else c.pre
    with pytest.raises(ValueError, match=name):
        getattr(binding, f"prefill_attn_varlen_{call}")(**t, scale=c.scale, **kw)


@pytest.mark.parametrize("name", ["prefix_v", "prefix_k_scale", "prefix_v_scale"])
def test_prefix_refuses_other_shapes_of_as_many_elements(name):
    c = Call(311, [3, 5], [20, 7], 64, 2, 2, int8="scale" in name, prefix=40)
    c.pre[name] = swapped(c.pre[name])
    with pytest.raises(ValueError, match=name):
        c.prefix()


@pytest.mark.parametrize("name", ["lse", "weights"])
def test_key_weights_refuses_other_shapes_of_as_many_elements(name):
    c = Call(312, [3, 5], [20, 7], 64, 2, 2)
    t = dict(lse=torch.zeros((8, 4), device="cuda"), weights=c.weights.cuda())
    t[name] = swapped(t[name])
    with pytest.raises(ValueError, match=name):
        binding.prefill_attn_key_weights(c.dev[0], c.dev[1], *c.meta, c.data[0][1], c.offsets, **t)


@pytest.mark.parametrize("name", ["cache_v", "weights", "kept_index", "kept_weights"])
def test_evict_refuses_other_shapes_of_as_many_elements(name):
    c = Call(313, [0] * 3, [90, 20, 60], 64, 2, 1)
    t = dict(cache_k=c.data[0][1], cache_v=c.data[1][1], weights=c.weights.cuda(), lengths=c.offsets,
             kept_lengths=torch.zeros_like(c.offsets), kept_weights=c.weights.cuda(),
             kept_index=torch.zeros((3, 2, 50), dtype=torch.int32, device="cuda"))
    t[name] = swapped(t[name])
    with pytest.raises(ValueError, match=name):
        binding.prefill_attn_evict(**t, budget=50)


# --------------------------------------------------------------------------- eviction: what a CTA selects from alone

@pytest.mark.parametrize("kept", ["new", "same"])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 1), (500, 4, 100), (2046, 0, 3), (2047, 3, 0), (2048, 4, 1000), (2049, 1, 1)])
def test_evict_at_the_length_that_one_launch_selects_alone(budget, sinks, recent, kept):
    """One launch: a CTA selects from up to 2048 tokens alone (its list is full at 2048 kept), its cluster from more."""
    for d, int8, block in ((64, False, 0), (32, True, 16)):
        c = Call(320, [0] * 3, [2047, 2048, 2049], d, 2, 1, block, int8)
        evict(c, weights_for(c, 1, "ties" if d == 64 else "special"), budget, sinks, recent, kept=kept)
        assert binding.prefill_attn_last_launch_count() == 1
    ok()


@pytest.mark.parametrize("kept", ["new", "same"])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 1), (500, 4, 100), (4095, 0, 3), (4096, 4, 1000), (4097, 1, 1)])
def test_evict_at_the_length_that_two_launches_select_alone(budget, sinks, recent, kept):
    """Two launches: a CTA selects from up to 4096 tokens alone, its cluster from more; a capacity of 4096 has no cluster."""
    for lens, slack in (([4095, 4096, 4097], 3), ([4096, 4095, 4096], 0)):
        c = Call(321, [0] * 3, lens, 32, 60, 1, slack=slack)
        evict(c, weights_for(c, 2, "special" if slack else "ties"), budget, sinks, recent, kept=kept)
        assert binding.prefill_attn_last_launch_count() == 2
    ok()


# --------------------------------------------------------------------------- what the attention calls leave in the cache

def rows_written(c, skipped=()):
    """[slots, heads, rows] of the cache: whether a sequence's new token has its row there; and the tokens of those rows
    in the order that the mask picks them."""
    at = torch.full(c.cache.shape[:-1], -1, dtype=torch.long)
    for b, (n, p) in enumerate(zip(c.new, c.lens)):
        if b in skipped:
            continue
        slot, row = c.cache.at(b, torch.arange(p, p + n))
        at[slot, :, row] = torch.arange(c.cu[b], c.cu[b + 1])[:, None]
    return at >= 0, at


def check_cache(c, w, new, tol, skipped=()):
    """K (w = 0) or V (1): the new tokens' rows within tol of `new` [tokens, heads, d] (None: the documented write, bit
    for bit), every other row as it was."""
    got, was = c.data[w][1].cpu(), c.cache.data[w]
    here, token = rows_written(c, skipped)
    assert torch.equal(R.bits(got)[~here], R.bits(was)[~here]), "a row that holds no new token was written"
    sc = None if c.sc[w] is None else c.sc[w][1].cpu()
    if sc is not None:
        assert torch.equal(R.bits(sc)[~here], R.bits(c.cache.scale[w])[~here]), "a scale of no new token was written"
    if tol is None:
        data, scale = c.cache.written(w, new, c.cu)
        assert torch.equal(R.bits(got)[here], R.bits(data)[here])
        assert sc is None or torch.equal(R.bits(sc)[here], R.bits(scale)[here])
        return
    head = torch.arange(c.hk)[None, :, None].expand(here.shape)[here]
    ref, tol = new[token[here], head].double(), tol[token[here], head].double()
    x = got[here].double()
    if sc is not None:
        step = sc[here].double()[:, None]
        most = ref.abs().amax(-1, keepdim=True)
        assert ((step * 127 - most).abs() <= tol.amax(-1, keepdim=True) + most * 2.0 ** -22).all(), "scale"
        x, tol = x * step, tol + step * (0.5 + 2.0 ** -10)  # and half a step of the code
    err = (x - ref).abs()
    assert (err <= tol).all(), f"off by {(err / tol).max():.2f} of the tolerance"


@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("call,new,lens", [("sinks", [3, 40, 0, 1], [300, 0, 9, 77]), ("prefix", [2, 17, 0, 130], [100, 0, 9, 31]),
                                           ("prefix", [1, 1], [64, 3])])
def test_rotary_keys_in_the_cache(call, new, lens, int8, block):
    """The cache gets the keys rotated to their absolute positions, behind the shared prefix's, and the values as given.

    Tolerance: the library's angle is position * inv_freq in fp32, inv_freq by a division and a power that may each be
    an ulp off the reference's, so an angle is within position * 2^-22 of it; a rotated value a cos - b sin moves by at
    most (|a| + |b|) times that and by its own fp32 roundings, (|a| + |b|) 2^-21; then both round to bf16, where two
    neighbours may be picked: a spacing, 2^-7 of the value.
    """
    theta, pre = 1e4, 150 if call == "prefix" else 0
    c = Call(330, new, lens, 64, 2, 2, block, int8, pre)
    c.sinks(90, 4, theta=theta) if call == "sinks" else c.prefix(theta=theta)
    torch.cuda.synchronize()
    c.guards()
    pos = torch.cat([torch.arange(n) + p + pre for n, p in zip(new, lens)])
    want = R.rotate(c.k, pos, theta)
    a, b = c.k.double().abs().chunk(2, -1)
    tol = 2.0 ** -7 * want.double().abs() + (a + b).repeat(1, 1, 2) * (pos.double()[:, None, None] * 2.0 ** -22 + 2.0 ** -21)
    # the test can tell: neither the key as given nor the one at the position without the prefix would pass
    for other in (c.k, R.rotate(c.k, pos - pre, theta) if pre else c.k, R.rotate(c.k, pos + 1, theta)):
        moved = pos > 0
        assert ((other.double() - want.double()).abs() > tol)[moved].any(-1).float().mean() > 0.9
    check_cache(c, 0, want, tol)
    check_cache(c, 1, c.v, None)
    ok()


@pytest.mark.parametrize("block", [0, 32])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("call", ["sinks", "prefix"])
def test_skipped_sequences_leave_the_other_caches_written(call, int8, block):
    """One sequence's metadata is inconsistent: the others' new rows are written, and nothing else."""
    c = Call(331, [1, 3, 40, 2], [20, 7, 200, 0], 64, 2, 2, block, int8, prefix=40 if call == "prefix" else 0)
    c.offsets[1] = 8  # disagrees with cu_seqlens_k
    c.sinks(64, 4) if call == "sinks" else c.prefix()
    torch.cuda.synchronize()
    c.guards()
    for w, new in ((0, c.k), (1, c.v)):
        check_cache(c, w, new, None, skipped=[1])
    assert binding.prefill_attn_device_status() == binding.DEVERR_METADATA


# --------------------------------------------------------------------------- precision of the key weights

@pytest.mark.parametrize("new,lens,d,group,block,int8", [
    ([2000], [0], 128, 1, 0, False),                   # 16 Q tiles under one key
    ([700, 90], [300, 0], 64, 4, 16, False),
    ([700, 90], [300, 0], 64, 4, 0, True),
    ([1] * 6, [900, 17, 0, 128, 300, 64], 128, 8, 0, False),
    ([1, 2, 30], [900, 17, 300], 32, 4, 32, True),
    ([150, 3], [40, 500], 64, 48, 0, False),           # 96 of a Q tile's 128 columns: bounds tested in every column
])
def test_key_weights_to_fp32(new, lens, d, group, block, int8):
    """Scores that fp32 holds exactly (q and k of -1, 0 and 1, or int8 codes), so that what is left is the exponent's
    argument, the exponential and the sum.

    In units of 2^-24, relative to a term: the argument x - l (in powers of two) has the roundings of log2(e), of its
    products with the scale, a row's scale and lse, and its own, at most 4 |x| + 3 |l| (of which ln 2 reaches the
    term); ex2.approx is within 4 of its result.  The sum of positive terms: chains of at most 64 columns of a Q tile,
    joined, then one addition per Q tile and at most three more: 70 + tiles.
    """
    c = Call(340, new, lens, d, 2, group, block, int8)
    g = torch.Generator().manual_seed(9)
    ints = lambda x: torch.randint(-1, 2, x.shape, generator=g).to(x.dtype)  # noqa: E731
    c.q, c.k, c.scale = ints(c.q), ints(c.k), 0.125
    c.dev[0].copy_(c.q), c.dev[1].copy_(c.k)
    if not int8:
        data = c.cache.data[0]
        c.cache.data[0] = torch.where(data.isnan(), data, ints(data))
        c.data[0][1].copy_(c.cache.data[0])
    lse = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale)[1].float()
    w = c.weights.cuda()
    binding.prefill_attn_key_weights(c.dev[0], c.dev[1], *c.meta, c.data[0][1], c.offsets, lse.cuda(), w, scale=c.scale,
                                     cache_k_scale=c.scales["cache_k_scale"], **c.opts)
    ref = R.key_weights(c.cache, c.q, c.k, c.new, lse, c.scale, c.weights)
    keys = c.k.double().norm(dim=-1).max()
    for b in range(len(lens)):
        if lens[b]:
            keys = max(keys, c.cache.logical(0, b).norm(dim=-1).max())
    x = math.log2(math.e) * c.scale * float(c.q.double().norm(dim=-1).max() * keys)  # |q . k| <= |q| |k|
    l2 = math.log2(math.e) * float(lse.abs().max())
    tiles = max(-(-n // (128 // group)) for n in new)
    tol = 2.0 ** -24 * (math.log(2) * (4 * x + 3 * l2) + 4 + 70 + tiles) * ref.abs() + 1e-30
    assert tol.max() / ref.abs().max() < 2.0 ** -14
    err = (w.cpu().double() - ref).abs()
    assert (err <= tol).all(), f"off by {(err / tol).max():.2f} of the tolerance"
    ok()


# --------------------------------------------------------------------------- precision of the attention over int8 caches

@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("call", ["sinks", "prefix"])
def test_int8_attention_rounds_twice(call, d, block):
    """P and the output are rounded to bf16, the values of an int8 cache are not.

    Roundings are independent, so their squares add, in 2-norms relative to the output.  r is that of the output
    alone, taken from the exact one; P's share is that of values spread over a binade, about 0.00153^2, against r^2 of
    about 0.00165^2: two roundings come to 1.9 r^2, and a third of the values to 2.7 r^2.
    """
    new, lens = [40, 1, 3], [700, 1500, 333]
    c = Call(350, new, lens, d, 2, 4, block, True, prefix=900 if call == "prefix" else 0)
    kw = dict(window=600, sinks=70) if call == "sinks" else {}
    c.sinks(600, 70) if call == "sinks" else c.prefix()
    c.check(**kw)
    ref, _, _ = R.attention(c.cache, c.q, c.k, c.v, c.new, c.scale, **kw)
    r = ((ref.to(torch.bfloat16).double() - ref).norm() / ref.norm()).item()
    err = ((c.out[1].cpu().double() - ref).norm() / ref.norm()).item()
    assert 0.0013 < r < 0.0019
    assert err ** 2 <= 2.3 * r ** 2, f"{err:.5f}: {(err / r) ** 2:.2f} of the output's rounding"
    ok()
