"""Host threads that call on one stream at the same time: the kernels of a call hand data to one another
through the stream's workspace, so each call's launches stay together."""
import threading

import pytest
import torch

from prefill_phase_attention_gb300 import binding
from tests import long_reference as R
from tests.test_long_context_gpu import Call, run_all, same, tensors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from prefill_phase_attention_gb300 import build
    build.build()
    binding.load()


def test_threads_on_one_stream_get_the_bits_of_calls_in_turn():
    """Four threads, each with sizes of its own (a scheduler of its own, rows cut into pieces, none), so that a list
    or partial result of another thread's call would show, on a workspace that grows as they go."""
    st = torch.cuda.Stream()
    made = [([1, 40, 0, 3], [300, 10, 5, 128]), ([1], [4000]), ([1] * 70, [60 + 7 * i for i in range(70)]),
            ([200, 1, 33], [0, 900, 77])]
    cs = [Call(200 + i, new, lens, 64, 2, 2, prefix=150 + 400 * i) for i, (new, lens) in enumerate(made)]
    wants = [tensors(c) for c in cs]
    for c, w in zip(cs, wants):
        run_all(c, w)  # one after the other, on the default stream
        binding.prefill_attn_varlen_ex(w["q"], w["k"], w["v"], *c.meta, w["ck"], w["cv"], c.offsets, w["out"], w["lse"],
                                       scale=c.scale, rope_theta=1e4)
    torch.cuda.synchronize()
    rounds, failed = 12, []
    got = [[tensors(c) for _ in range(rounds)] for c in cs]
    torch.cuda.synchronize()
    start = threading.Barrier(len(cs))

    def work(c, runs):
        try:
            with torch.cuda.stream(st):
                start.wait()
                for d in runs:
                    run_all(c, d, st)
                    binding.prefill_attn_varlen_ex(d["q"], d["k"], d["v"], *c.meta, d["ck"], d["cv"], c.offsets,
                                                   d["out"], d["lse"], scale=c.scale, rope_theta=1e4, stream=st)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(cs, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for want, runs in zip(wants, got):
        for d in runs:
            same(d, want)
    assert R.bits(got[0][0]["out"]).any()
    with torch.cuda.stream(st):
        assert binding.prefill_attn_device_status(st) == 0
    assert binding.prefill_attn_device_status() == 0
