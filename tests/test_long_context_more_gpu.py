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
