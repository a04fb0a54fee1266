"""More GPU tests of the long-context calls: sizes, options and argument shapes at their edges."""
import pytest
import torch

from prefill_phase_attention_gb300 import binding
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
