"""GPU tests of the 4-bit cache at the edges of its calls' documented range, against the plain 64-bit forms and error
bounds of tests/cache4_reference.py."""
import math

import pytest
import torch

from prefill_phase_attention_gb300 import binding
from tests import cache4_reference as R
from tests.test_cache4_gpu import Call, DIMS

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from prefill_phase_attention_gb300 import build
    build.build()
    binding.load()
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need CUDA")


# ---------------------------------------------------------------------------
# row blocks of one tile (nothing cached that is visible, at most 8 new tokens), several in a row in one warp's share
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 5, 8])
@pytest.mark.parametrize("d,group", DIMS)
def test_empty_caches_beside_long_ones(d, group, n):
    """Long decode rows make the shares long; sequences with nothing cached stand in the middle and at the end."""
    c = Call(1, [1] * 8 + [n] * 6 + [1] * 8 + [n] * 2, [8192] * 8 + [0] * 6 + [8192] * 8 + [0] * 2, d, hk=2, share=64,
             group=group)
    c.attend()
    assert not c.expanded
    c.check()


@pytest.mark.parametrize("past,window", [(0, 0), (96, 1)])
@pytest.mark.parametrize("seqs,block", [(256, 16), (300, 0)])
@pytest.mark.parametrize("d,group", [(128, 128), (128, 64), (128, 32), (64, 32), (32, 32)])
def test_many_rows_without_cached_keys(d, group, seqs, block, past, window):
    """As many sequences as a CTA keeps in shared memory, and more; a window of one token hides whole tiles."""
    c = Call(2, [1] * seqs, [past] * seqs, d, hk=4, share=128, group=group, block=block)
    c.attend(window=window)
    assert not c.expanded
    c.check(window=window)
