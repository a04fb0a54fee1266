"""What a stream's workspace keeps once a graph was captured on the stream."""
import ctypes

import pytest
import torch

from prefill_phase_attention_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from prefill_phase_attention_gb300 import build
    build.build()
    binding.load()


def pool_bytes():
    """Bytes that the device's default memory pool holds, which the workspaces come from (torch's tensors do not).
    A synchronisation gives back what is free of it."""
    torch.cuda.synchronize()
    cuda = ctypes.CDLL("libcuda.so.1")
    dev, pool, held = ctypes.c_int(), ctypes.c_void_p(), ctypes.c_uint64()
    assert cuda.cuDeviceGet(ctypes.byref(dev), torch.cuda.current_device()) == 0
    assert cuda.cuDeviceGetDefaultMemPool(ctypes.byref(pool), dev) == 0
    reserved_mem_current = 5
    assert cuda.cuMemPoolGetAttribute(pool, reserved_mem_current, ctypes.byref(held)) == 0
    return held.value


class Sizes:
    """A call of one sequence of up to `most` tokens; run(t, st) makes it with the first t of them."""

    def __init__(self, most, H=8, hk=2, d=128):
        mk = lambda *s: torch.randn(s, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.q, self.k, self.v, self.out = mk(most, H, d), mk(most, hk, d), mk(most, hk, d), mk(most, H, d)
        self.ck, self.cv = mk(1, hk, most, d), mk(1, hk, most, d)
        self.pre = mk(hk, 64, d), mk(hk, 64, d)
        self.zero = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lse = torch.zeros((most, H), device="cuda")
        self.cu = {t: torch.tensor([0, t], dtype=torch.int32, device="cuda") for t in range(0, most + 1, 500)}

    def run(self, t, st, call):
        args = (self.q[:t], self.k[:t], self.v[:t], self.cu[t], self.cu[t], self.ck, self.cv, self.zero, self.out[:t],
                self.lse[:t])
        if call == "rotary":
            binding.prefill_attn_varlen_ex(*args, rope_theta=1e4, stream=st)
        else:
            binding.prefill_attn_varlen_prefix(*args, prefix_k=self.pre[0], prefix_v=self.pre[1], stream=st)


@pytest.mark.parametrize("call", ["rotary", "prefix"])
def test_workspaces_that_a_graph_outgrew_are_bounded(call):
    """Forty ever longer prompts on a stream that a graph was captured on: the blocks that the graph may use stay,
    and what stays is bounded by a few times the largest call's need, not by the sum of them all."""
    most = 40 * 500
    s, st = Sizes(most), torch.cuda.Stream()
    binding.prefill_attn_release()
    free = pool_bytes()
    with torch.cuda.stream(st):
        s.run(most, st, call)
    need = pool_bytes() - free  # of the largest call
    binding.prefill_attn_release()
    assert pool_bytes() == free
    with torch.cuda.stream(st):
        s.run(500, st, call)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        s.run(500, st, call)
    with torch.cuda.stream(st):
        s.run(500, st, call)
    want = s.out[:500].clone()
    for t in range(1000, most + 1, 500):
        with torch.cuda.stream(st):
            s.run(t, st, call)
    kept = pool_bytes() - free
    assert kept <= 4 * need, f"{kept >> 20} MiB are kept, {kept / need:.1f} times the largest call's {need >> 20}"
    s.out.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out[:500], want) and binding.prefill_attn_device_status(st) == 0
    del g
    binding.prefill_attn_release()
    assert pool_bytes() == free
