"""The 4-bit cache's calls reject argument errors before touching a GPU, and its plain form keeps the format (CPU tests)."""
import ctypes

import pytest
import torch

from prefill_phase_attention_gb300 import binding, build
from tests import cache4_reference as R
from tests.test_long_context_abi import options, refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


FAR = {name: (i + 1) << 32 for i, name in enumerate(["q", "k", "v", "cu_q", "cu_k", "off", "out", "lse", "ck", "cv", "kp", "vp"])}


def cache(kw):
    if kw.get("cache", 0) is None:
        return None
    c = binding.PaCache4(ctypes.sizeof(binding.PaCache4), 64, FAR["ck"], FAR["cv"], FAR["kp"], FAR["vp"])
    for name, v in kw.get("c", {}).items():
        setattr(c, name, v)
    return ctypes.byref(c)


def attend(lib, **kw):
    a = dict({n: FAR[n] for n in ("q", "k", "v", "cu_q", "cu_k", "off", "out", "lse")}, num_seqs=1, total=4, cap=8, H=4,
             Hk=2, d=64, scale=0.125, causal=1)
    a.update({k: v for k, v in kw.items() if k in a})
    return lib.prefill_attn_varlen_cache4(a["q"], a["k"], a["v"], a["cu_q"], a["cu_k"], cache(kw), a["off"], a["out"],
                                          a["lse"], a["num_seqs"], a["total"], a["cap"], a["H"], a["Hk"], a["d"], a["scale"],
                                          a["causal"], ctypes.byref(options(**kw.get("o", {}))), None)


def copy(lib, which, **kw):
    a = dict(k=FAR["k"], v=FAR["v"], cu=FAR["cu_q"], off=FAR["off"], num_seqs=1, total=4, cap=8, Hk=2, d=64)
    a.update({k: v for k, v in kw.items() if k in a})
    sizes = (a["num_seqs"], a["total"], a["cap"], a["Hk"], a["d"], ctypes.byref(options(**kw.get("o", {}))), None)
    if which == "write":
        return lib.prefill_attn_cache4_write(a["k"], a["v"], a["cu"], cache(kw), a["off"], *sizes)
    return lib.prefill_attn_cache4_read(cache(kw), a["cu"], a["off"], a["k"], a["v"], *sizes)


PAGED = dict(block_table=1 << 50, block_size=8, max_blocks_per_seq=1, num_blocks=4)

SHARED = [
    (dict(cache=None), 1, "cache is NULL"),
    (dict(c=dict(struct_size=8)), 1, "struct_size"),
    (dict(c=dict(group=48)), 1, "group"),
    (dict(c=dict(group=128)), 1, "group"),
    (dict(c=dict(k=None)), 1, "pa_cache4.k is NULL"),
    (dict(c=dict(v_params=FAR["vp"] + 8)), 1, "16-byte"),
    (dict(c=dict(k_params=FAR["k"])), 1, "overlap"),
    (dict(k=FAR["k"] + 2), 1, "16-byte"),
    (dict(d=48), 2, "head_dim"),
    (dict(num_seqs=-1), 1, "num_seqs"),
    (dict(cap=0), 1, "max_cache_len"),
    (dict(cap=2 ** 30 + 1, Hk=1, H=1), 2, "2^30"),
    (dict(num_seqs=2 ** 30 + 1, Hk=1, H=1, cap=1), 2, "2^30"),
    (dict(o=dict(kv_quant=1, cache_k_scale=512, cache_v_scale=1024)), 1, "kv_quant"),
    (dict(o=dict(schedule=2)), 1, "schedule"),
    (dict(o=dict(wait_timeout_test=1)), 1, "wait_timeout_test"),
    (dict(o=dict(PAGED, block_size=16)), 1, "max_cache_len"),
    (dict(o=dict(PAGED, block_size=12), cap=12), 2, "block_size"),
    (dict(o=dict(PAGED, num_blocks=2 ** 28)), 2, "2^32"),
]


@pytest.mark.parametrize("kw,status,msg", SHARED + [
    (dict(q=None), 1, "q is NULL"),
    (dict(lse=FAR["lse"] + 2), 1, "4-byte"),
    (dict(out=FAR["q"] + 64), 1, "overlap"),
    (dict(lse=FAR["cu_q"]), 1, "overlap"),
    (dict(H=5), 1, "multiple"),
    (dict(scale=0.0), 1, "scale"),
    (dict(causal=0, o=dict(window=4)), 1, "causal"),
    (dict(o=dict(window=-1)), 1, "window"),
])
def test_attend_refusals(lib, kw, status, msg):
    refused(lib, attend(lib, **kw), status, msg)


@pytest.mark.parametrize("which", ["write", "read"])
@pytest.mark.parametrize("kw,status,msg", SHARED + [
    (dict(v=None), 1, "v is NULL"),
    (dict(cu=FAR["cu_q"] + 1), 1, "4-byte"),
    (dict(total=-1), 1, "total"),
    (dict(Hk=0), 1, "n_kv_heads"),
    (dict(total=2 ** 29, Hk=2), 2, "2^30"),
    (dict(o=dict(window=4)), 1, "window"),
])
def test_copy_refusals(lib, which, kw, status, msg):
    refused(lib, copy(lib, which, **kw), status, msg)


def test_caches_that_are_written_do_not_overlap(lib):
    """(64 channels, 16 rows: 512 bytes of codes)"""
    refused(lib, attend(lib, c=dict(v=FAR["ck"] + 512 - 16)), 1, "overlap")
    refused(lib, copy(lib, "write", c=dict(v=FAR["ck"] + 512 - 16)), 1, "overlap")


def test_read_takes_no_rotation_and_no_aliases(lib):
    refused(lib, copy(lib, "read", o=dict(rope_theta=1e4)), 1, "rope_theta")
    refused(lib, copy(lib, "read", v=FAR["k"]), 1, "overlap")
    refused(lib, copy(lib, "read", k=FAR["cu_q"]), 1, "overlap")


def test_empty_calls_are_no_ops(lib):
    for kw in (dict(num_seqs=0), dict(total=0)):
        nothing = dict(c=dict(k=None, v=None, k_params=None, v_params=None), **kw)
        assert attend(lib, q=None, k=None, v=None, out=None, **nothing) == 0
        for which in ("write", "read"):
            assert copy(lib, which, k=None, v=None, **nothing) == 0
    assert lib.prefill_attn_last_launch_count() == 0


def test_python_checks_need_no_gpu():
    x = torch.zeros((2, 2, 64), dtype=torch.bfloat16)
    c, p = torch.zeros((1, 2, 8, 32), dtype=torch.uint8), torch.zeros((1, 2, 8, 1, 2), dtype=torch.bfloat16)
    cu, off = torch.tensor([0, 2], dtype=torch.int32), torch.tensor([0], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        binding.prefill_attn_cache4_write(x, x, cu, c, c, off, cache_k_params=p, cache_v_params=p)
    with pytest.raises(ValueError, match="CUDA"):
        binding.prefill_attn_varlen_cache4(x, x, x, cu, cu, c, c, off, x, cache_k_params=p, cache_v_params=p)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_the_plain_format_holds_its_error(group):
    g = torch.Generator().manual_seed(0)
    x = (torch.randn((500, 128), generator=g) * torch.rand((500, 1), generator=g) * 9).to(torch.bfloat16)
    codes, params = R.quantise(x, group)
    y = x.double().unflatten(-1, (-1, group))
    span = (y.amax(-1) - y.amin(-1))[..., None]
    err = (R.values(codes, params).unflatten(-1, (-1, group)) - y).abs()
    # half a step of a scale that is off by 2^-8, and 15 steps of that rounding at the top
    assert (err <= span / 30 * (1 + R.U) + span * R.U + 1e-9).all()
    assert torch.equal(params[..., 1].float(), y.amin(-1).float())
