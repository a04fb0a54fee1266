"""More argument errors that the long-context calls report before touching a GPU (CPU tests)."""
import ctypes

import pytest
import torch

from prefill_phase_attention_gb300 import binding, build
from tests.test_long_context_abi import options, refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def attention(**kw):
    """Arguments of an attention call from q on, up to the scale: tensors far from one another, one sequence."""
    a = dict(q=1 << 30, k=2 << 30, v=3 << 30, cu_q=64, cu_k=256, ck=4 << 30, cv=5 << 30, off=512, out=6 << 30, lse=None,
             num_seqs=1, total_q=4, cap=8, H=4, Hk=2, d=64, scale=0.125)
    a.update(kw)
    return list(a.values())


def key_weights(**kw):
    a = dict(q=1 << 30, k=2 << 30, cu_q=64, cu_k=256, ck=4 << 30, off=512, lse=7 << 30, weights=8 << 30, num_seqs=1,
             total_q=4, cap=8, H=4, Hk=2, d=64, scale=0.125, causal=1, sinks=0, prefix=0)
    a.update(kw)
    return list(a.values())


def prefix(**kw):
    p = binding.PaPrefix(ctypes.sizeof(binding.PaPrefix), 5, 9 << 30, 10 << 30, 8, 0, None, None, None)
    for name, v in kw.items():
        setattr(p, name, v)
    return ctypes.byref(p)


@pytest.mark.parametrize("paged", [False, True])
def test_more_sequences_than_the_schedulers_count(lib, paged):
    """Their loops step 1024 sequences at a time in 32 bits: near 2^31 sequences a step would pass the end of int."""
    n = 2 ** 30 + 1
    o = dict(block_table=1 << 40, block_size=8, max_blocks_per_seq=1, num_blocks=4) if paged else {}
    sizes = dict(num_seqs=n, total_q=1, H=1, Hk=1, cap=8 if paged else 1)
    refused(lib, lib.prefill_attn_varlen_sinks(*attention(**sizes), 2, ctypes.byref(options(4, **o)), None), 2, "num_seqs")
    p = prefix(block_table=1 << 41, len=1, capacity=1)
    refused(lib, lib.prefill_attn_varlen_prefix(*attention(**sizes), 1, p, ctypes.byref(options(0, **o)), None), 2, "num_seqs")
    refused(lib, lib.prefill_attn_key_weights(*key_weights(**sizes), ctypes.byref(options(0, **o)), None), 2, "num_seqs")


EVICT = dict(ck=1 << 25, cv=1 << 26, weights=1 << 24, lengths=1 << 20, new=1 << 21, index=1 << 22, kept_w=1 << 23,
             num_seqs=2, cap=64, Hk=2, d=64, budget=6, sinks=1, recent=2)
CODES = dict(kv_quant=1, cache_k_scale=1 << 27, cache_v_scale=1 << 28)


# 256 rows of fp32 weights or scales (1024 bytes) and of 128 bytes of keys and values (32 KiB; int8: 16 KiB)
@pytest.mark.parametrize("kw,o,msg", [
    (dict(new=(1 << 24) + 1020), {}, "kept_lengths must not overlap weights"),
    (dict(new=(1 << 23) + 4), {}, "kept_lengths must not overlap kept_weights"),
    (dict(new=(1 << 25) + 32764), {}, "kept_lengths must not overlap cache_k"),
    (dict(lengths=(1 << 26) + 32764), {}, "cache_v must not overlap lengths"),
    (dict(lengths=(1 << 23) + 1020), {}, "kept_weights must not overlap lengths"),
    (dict(index=(1 << 25) - 8), {}, "kept_index must not overlap cache_k"),
    (dict(kept_w=(1 << 26) - 1020), {}, "kept_weights must not overlap cache_v"),
    (dict(weights=(1 << 25) - 1020), {}, "cache_k must not overlap weights"),
    (dict(index=(1 << 27) + 1020), CODES, "kept_index must not overlap cache_k_scale"),
    (dict(kept_w=(1 << 28) + 1020), CODES, "kept_weights must not overlap cache_v_scale"),
    (dict(), dict(CODES, cache_v_scale=(1 << 27) + 1020), "cache_k_scale must not overlap cache_v_scale"),
    (dict(weights=(1 << 27) - 1020), CODES, "cache_k_scale must not overlap weights"),
    (dict(new=1 << 30), dict(block_table=(1 << 30) + 4, block_size=8, max_blocks_per_seq=8, num_blocks=16),
     "kept_lengths must not overlap block_table"),
])
def test_evict_refuses_overlapping_buffers(lib, kw, o, msg):
    a = list({**EVICT, **kw}.values())
    refused(lib, lib.prefill_attn_evict(*a, ctypes.byref(options(0, **o)), None), 1, msg)


# q 4 x 4 heads x 128 bytes, k 4 x 2 x 128, lse 4 x 4 floats, weights 2 x 8 floats, cached keys 2 x 8 x 128 (int8: 64)
@pytest.mark.parametrize("kw,o,msg", [
    (dict(weights=(1 << 30) + 2044), {}, "weights must not overlap q"),
    (dict(weights=(2 << 30) - 60), {}, "weights must not overlap k"),
    (dict(weights=(4 << 30) + 2044), {}, "weights must not overlap cache_k"),
    (dict(weights=(7 << 30) + 60), {}, "weights must not overlap lse"),
    (dict(weights=(7 << 30) - 60), {}, "weights must not overlap lse"),
    (dict(weights=68), {}, "weights must not overlap cu_seqlens_q"),
    (dict(weights=260), {}, "weights must not overlap cu_seqlens_k"),
    (dict(weights=512), {}, "weights must not overlap cache_offsets"),
    (dict(weights=(11 << 30) + 60), dict(kv_quant=1, cache_k_scale=11 << 30, cache_v_scale=12 << 30),
     "weights must not overlap cache_k_scale"),
    (dict(weights=(11 << 30) - 124), dict(block_table=11 << 30, block_size=8, max_blocks_per_seq=1, num_blocks=2),
     "weights must not overlap block_table"),
])
def test_key_weights_refuses_overlapping_buffers(lib, kw, o, msg):
    refused(lib, lib.prefill_attn_key_weights(*key_weights(**kw), ctypes.byref(options(0, **o)), None), 1, msg)


# out 4 x 4 heads x 128 bytes, lse 4 x 4 floats; of the prefix 8 + 5 rows of 128 bytes (int8: 64 and a scale)
@pytest.mark.parametrize("kw,p,o,msg", [
    (dict(), dict(k=(6 << 30) + 2032), {}, "out must not overlap the prefix's k"),
    (dict(), dict(v=(6 << 30) - 13 * 128 + 16), {}, "out must not overlap the prefix's v"),
    (dict(lse=(9 << 30) + 13 * 128 - 4), {}, {}, "lse must not overlap the prefix's k"),
    (dict(lse=(10 << 30) - 60), {}, {}, "lse must not overlap the prefix's v"),
    (dict(lse=13 << 30), dict(k_scale=(13 << 30) + 60, v_scale=14 << 30),
     dict(kv_quant=1, cache_k_scale=11 << 30, cache_v_scale=12 << 30), "lse must not overlap the prefix's k_scale"),
    (dict(), dict(k_scale=13 << 30, v_scale=(6 << 30) - 48),
     dict(kv_quant=1, cache_k_scale=11 << 30, cache_v_scale=12 << 30), "out must not overlap the prefix's v_scale"),
    (dict(), dict(block_table=(6 << 30) + 2044), dict(block_table=256, block_size=8, max_blocks_per_seq=1, num_blocks=4),
     "out must not overlap the prefix's block_table"),
])
def test_prefix_refuses_overlapping_buffers(lib, kw, p, o, msg):
    got = lib.prefill_attn_varlen_prefix(*attention(**kw), 1, prefix(**p), ctypes.byref(options(0, **o)), None)
    refused(lib, got, 1, msg)


@pytest.mark.parametrize("kw,msg", [
    (dict(block_table="t", prefix_table="t", prefix_len=3, prefix_k="x"), "prefix_k"),
    (dict(block_table="t", prefix_table="t", prefix_len=3, prefix_v="x"), "prefix_v"),
    (dict(block_table="t", prefix_table="t", prefix_len=3, prefix_k_scale="x"), "prefix_k_scale"),
    (dict(block_table="t", prefix_table="t", prefix_len=3, prefix_v_scale="x"), "prefix_v_scale"),
    (dict(prefix_k="x", prefix_v="x", prefix_table="t"), "prefix_table"),
    (dict(prefix_k="x", prefix_v="x", prefix_k_scale="x"), "prefix_k_scale"),
    (dict(prefix_k="x", prefix_v="x", prefix_v_scale="x"), "prefix_v_scale"),
])
def test_binding_refuses_a_prefix_of_the_other_kind_of_cache(lib, kw, msg):
    """A prefix tensor that the call would not read is an error, not ignored."""
    x, t = torch.zeros(4, 2, 32, dtype=torch.bfloat16), torch.zeros((1, 2), dtype=torch.int32)
    kw = {n: {"x": x, "t": t}.get(v, v) if isinstance(v, str) else v for n, v in kw.items()}
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match=msg):
        binding.prefill_attn_varlen_prefix(x, x, x, i, i, x[None], x[None], i[:1], x, **kw)
