"""The long-context calls reject host-checkable argument errors before touching a GPU (CPU tests)."""
import ctypes

import pytest
import torch

from prefill_phase_attention_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def options(window=0, **kw):
    o = binding.PaOptions()
    o.struct_size = ctypes.sizeof(o)
    o.window = window
    for k, v in kw.items():
        setattr(o, k, v)
    return o


PAGED = dict(block_table=256, block_size=8, max_blocks_per_seq=1, num_blocks=4)
QUANT = dict(kv_quant=1, cache_k_scale=512, cache_v_scale=1024)


def refused(lib, status, want, msg):
    assert status == want, lib.prefill_attn_last_error()
    assert msg in lib.prefill_attn_last_error().decode()


def attention_args(kw):
    a = dict(q=16, k=32, v=48, cu_q=64, cu_k=80, ck=96, cv=112, off=128, out=144, lse=None, num_seqs=1, total_q=4,
             cap=8, H=4, Hk=2, d=64, scale=0.125)
    a.update({k: v for k, v in kw.items() if k in a})
    return list(a.values())


@pytest.mark.parametrize("kw,status,msg", [
    (dict(window=0), 1, "window"),
    (dict(window=-3), 1, "window"),
    (dict(sinks=-1), 1, "sink_tokens"),
    (dict(opts=None), 1, "window"),
    (dict(o=dict(wait_timeout_test=1)), 1, "wait_timeout_test"),
    (dict(o=dict(schedule=4)), 1, "schedule"),
    (dict(d=48), 2, "head_dim"),
    (dict(H=6, Hk=4), 1, "multiple"),
    (dict(scale=float("nan")), 1, "scale"),
    (dict(q=None), 1, "q is NULL"),
    (dict(out=16), 1, "alias"),
    (dict(o=dict(PAGED, block_size=16)), 1, "max_cache_len"),
    (dict(o=dict(QUANT, schedule=1)), 1, "schedule 1 needs"),
    (dict(cap=2 ** 30 + 1, H=1, Hk=1), 2, "2^30"),
])
def test_sinks_refusals(lib, kw, status, msg):
    opts = kw["opts"] if "opts" in kw else ctypes.byref(options(kw.get("window", 4), **kw.get("o", {})))
    refused(lib, lib.prefill_attn_varlen_sinks(*attention_args(kw), kw.get("sinks", 2), opts, None), status, msg)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(prefix=None), 1, "prefix is NULL"),
    (dict(p=dict(struct_size=8)), 1, "struct_size"),
    (dict(p=dict(reserved=1)), 1, "reserved"),
    (dict(p=dict(len=-1)), 1, "pa_prefix.len"),
    (dict(p=dict(len=9, capacity=8)), 1, "capacity"),
    (dict(p=dict(k=None)), 1, "must not be NULL"),
    (dict(p=dict(v=168)), 1, "16-byte"),
    (dict(p=dict(k=144)), 1, "alias"),
    (dict(o=dict(QUANT)), 1, "k_scale"),
    (dict(o=dict(QUANT), p=dict(k_scale=2050, v_scale=4096)), 1, "4-byte"),
    (dict(o=dict(PAGED)), 1, "pa_prefix.block_table"),
    (dict(o=dict(PAGED), p=dict(block_table=258)), 1, "4-byte"),
    (dict(o=dict(window=5)), 1, "window"),
    (dict(o=dict(wait_timeout_test=1)), 1, "wait_timeout_test"),
    (dict(d=40), 2, "head_dim"),
    (dict(causal=2), 1, "causal"),
    (dict(cap=2 ** 30 + 1, H=1, Hk=1), 2, "2^30"),
    (dict(p=dict(len=2 ** 30 + 1, capacity=2 ** 30 + 1)), 2, "2^30"),
    (dict(o=dict(PAGED), p=dict(len=2 ** 30 + 1, block_table=256)), 2, "2^30"),
])
def test_prefix_refusals(lib, kw, status, msg):
    p = binding.PaPrefix(ctypes.sizeof(binding.PaPrefix), 5, 160, 176, 8, 0, None, None, None)
    for name, v in kw.get("p", {}).items():
        setattr(p, name, v)
    ref = None if "prefix" in kw else ctypes.byref(p)
    got = lib.prefill_attn_varlen_prefix(*attention_args(kw), kw.get("causal", 1), ref,
                                         ctypes.byref(options(**kw.get("o", {}))), None)
    refused(lib, got, status, msg)


def test_prefix_layout_matches_header():
    P = binding.PaPrefix
    assert [(n, getattr(P, n).offset) for n, _ in P._fields_] == [
        ("struct_size", 0), ("len", 4), ("k", 8), ("v", 16), ("capacity", 24), ("reserved", 28), ("k_scale", 32),
        ("v_scale", 40), ("block_table", 48)]
    assert ctypes.sizeof(P) == 56


@pytest.mark.parametrize("kw,status,msg", [
    (dict(lse=None), 1, "lse is NULL"),
    (dict(weights=None), 1, "weights is NULL"),
    (dict(weights=162), 1, "4-byte"),
    (dict(weights=16), 1, "alias"),
    (dict(weights=96), 1, "alias"),
    (dict(sinks=-1, o=dict(window=4)), 1, "sink_tokens"),
    (dict(sinks=1), 1, "window"),
    (dict(prefix=-1), 1, "prefix_len"),
    (dict(prefix=3, o=dict(window=4)), 1, "window"),
    (dict(o=dict(schedule=2)), 1, "schedule"),
    (dict(o=dict(window=4), causal=0), 1, "causal"),
    (dict(d=48), 2, "head_dim"),
    (dict(q=None), 1, "q is NULL"),
    (dict(k=33), 1, "aligned"),
    (dict(o=dict(kv_quant=1, cache_k_scale=512)), 1, "cache_v_scale"),
    (dict(o=dict(PAGED, block_size=12)), 2, "power of two"),
    (dict(k=256, cap=2 ** 30 + 1, H=1, Hk=1), 2, "2^30"),
    (dict(k=256, prefix=2 ** 30 + 1), 2, "2^30"),
])
def test_key_weights_refusals(lib, kw, status, msg):
    a = dict(q=16, k=32, cu_q=64, cu_k=80, ck=96, off=128, lse=144, weights=160, num_seqs=1, total_q=4, cap=8, H=4, Hk=2,
             d=64, scale=0.125, causal=1, sinks=0, prefix=0)
    a.update({k: v for k, v in kw.items() if k in a})
    refused(lib, lib.prefill_attn_key_weights(*a.values(), ctypes.byref(options(**kw.get("o", {}))), None), status, msg)


@pytest.mark.parametrize("kw,status,msg", [
    (dict(budget=0), 1, "budget"),
    (dict(sinks=3, recent=4), 1, "fit the budget"),
    (dict(sinks=-1), 1, "fit the budget"),
    (dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), 1, "fit the budget"),
    (dict(num_seqs=-1), 1, "num_seqs"),
    (dict(cap=0), 1, "max_cache_len"),
    (dict(Hk=0), 1, "n_kv_heads"),
    (dict(d=16), 2, "head_dim"),
    (dict(num_seqs=2 ** 23, Hk=2), 2, "2^24"),
    (dict(num_seqs=2 ** 20, cap=2 ** 12), 2, "2^31"),
    (dict(num_seqs=1, Hk=1, cap=2 ** 30 + 1), 2, "2^30"),
    (dict(ck=None), 1, "cache_k is NULL"),
    (dict(cv=40), 1, "16-byte"),
    (dict(weights=None), 1, "weights is NULL"),
    (dict(lengths=1 << 20 | 2), 1, "4-byte"),
    (dict(new=1 << 20), 1, "kept_lengths must not overlap"),
    (dict(kept_w=(1 << 24) + 4), 1, "kept_weights must be"),
    (dict(index=2), 1, "4-byte"),
    (dict(index=(1 << 24) + 8), 1, "kept_index must not overlap"),
    (dict(index=1 << 21), 1, "kept_index must not overlap"),
    (dict(cv=1 << 25), 1, "cache_k and cache_v"),
    (dict(o=dict(window=4)), 1, "window"),
    (dict(o=dict(rope_theta=1e4)), 1, "rope_theta"),
    (dict(o=dict(schedule=1)), 1, "schedule"),
    (dict(o=dict(PAGED)), 1, "max_cache_len"),
])
def test_evict_refusals(lib, kw, status, msg):
    a = dict(ck=1 << 25, cv=1 << 26, weights=1 << 24, lengths=1 << 20, new=1 << 21, index=None, kept_w=None, num_seqs=2,
             cap=64, Hk=2, d=64, budget=6, sinks=1, recent=2)
    a.update({k: v for k, v in kw.items() if k in a})
    refused(lib, lib.prefill_attn_evict(*a.values(), ctypes.byref(options(**kw.get("o", {}))), None), status, msg)


def test_empty_batches_are_no_ops(lib):
    o = ctypes.byref(options(4))
    assert lib.prefill_attn_varlen_sinks(*attention_args(dict(num_seqs=0, q=None)), 2, o, None) == 0
    assert lib.prefill_attn_evict(None, None, None, None, None, None, None, 0, 8, 2, 64, 4, 0, 0, None, None) == 0
    assert lib.prefill_attn_key_weights(*[None] * 8, 0, 0, 8, 4, 2, 64, 0.125, 1, 0, 0, None, None) == 0
    assert lib.prefill_attn_last_launch_count() == 0


def test_bindings_refuse_cpu_tensors(lib):
    x = torch.zeros(4, 2, 32, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    w = torch.zeros(1, 4, 2)
    with pytest.raises(ValueError):
        binding.prefill_attn_varlen_sinks(x, x, x, i, i, x[None], x[None], i[:1], x, window=4, sink_tokens=1)
    with pytest.raises(ValueError):
        binding.prefill_attn_varlen_prefix(x, x, x, i, i, x[None], x[None], i[:1], x, prefix_k=x, prefix_v=x)
    with pytest.raises(ValueError):
        binding.prefill_attn_key_weights(x, x, i, i, x[None], i[:1], w[0], w)
    with pytest.raises(ValueError):
        binding.prefill_attn_evict(x[None], x[None], w, i[:1], i[:1].clone(), budget=2)


def test_bindings_refuse_integers_past_32_bits(lib):
    """ctypes would cut them off: 2^32 + 5 tokens of budget would become 5."""
    x = torch.zeros(4, 2, 32, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="sink_tokens"):
        binding.prefill_attn_varlen_sinks(x, x, x, i, i, x[None], x[None], i[:1], x, window=4, sink_tokens=1 << 32)
    with pytest.raises(ValueError, match="budget"):
        binding.prefill_attn_evict(x[None], x[None], torch.zeros(1, 4, 2), i[:1], i[:1].clone(), budget=(1 << 32) + 5)
