"""GPU tests of the 4-bit cache at the edges of its calls' documented range, against the plain 64-bit forms and error
bounds of tests/cache4_reference.py."""
import pytest
import torch

from prefill_phase_attention_gb300 import binding
from tests import cache4_reference as R
from tests.test_cache4_gpu import Call, DIMS, same_bits

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


# ---------------------------------------------------------------------------
# magnitudes
# ---------------------------------------------------------------------------

def shared_rows(seed, d=128, group=128, past=8192, seqs=16):
    """A call whose warps have shares of some 27 tiles: what one tile of a row block leaves meets the next ones."""
    return Call(seed, [1] * seqs, [past] * seqs, d, hk=2, share=64, group=group)


def scaled(c, which, factor):
    """Multiplies the parameters of a call's cached keys (0) or values (1)."""
    c.cache.params[which] = (c.cache.params[which].double() * factor).to(torch.bfloat16)
    c.params[which][1].copy_(c.cache.params[which])


def raised(c, nats):
    """Every 8th tile of 32 keys scores `nats` higher on average: queries are positive, the keys' minima grow by one
    number."""
    c.q = c.q.abs()
    c.dev[0].copy_(c.q)
    up = nats / (c.q.double().sum(-1).mean() * c.scale)
    later = torch.arange(c.cache.cap) // 32 % 8 == 7
    c.cache.params[0][..., 1] = (c.cache.params[0][..., 1].double() + up * later[:, None]).to(torch.bfloat16)
    c.params[0][1].copy_(c.cache.params[0])
    return later


@pytest.mark.parametrize("d,group", DIMS)
@pytest.mark.parametrize("nats,early,late", [
    (140, 45, 0),    # what came before the jump is 2^-157 of what comes after it
    (80, 60, 0),     # 2^-55
    (80, 90, -20),   # about as much
    (75, 90, 90),
    (80, -60, 40),
])
def test_jumps_of_the_maximum_between_values_of_any_size(d, group, nats, early, late):
    """The score rises by more than 100 in log2 units within a warp's share, values before and after differ by powers of 2."""
    c = shared_rows(3, d, group)
    later = raised(c, nats)
    scaled(c, 1, torch.where(later, 2.0 ** late, 2.0 ** early)[:, None, None].double())
    c.attend()
    assert not c.expanded
    c.check()


@pytest.mark.parametrize("past", [7, 40, 257])
def test_a_query_of_zeros_under_any_scale(past):
    """scale is any finite number above 0: a query of zeros weighs every visible key alike."""
    c = Call(4, [3, 1, 1], [past, 0, 1], hk=2, share=5, group=64)
    c.q[:, ::2] = 0
    c.dev[0].copy_(c.q)
    c.scale = 1e-20
    c.attend()
    c.check()


@pytest.mark.parametrize("d,group", [(128, 64), (128, 32), (64, 32)])
@pytest.mark.parametrize("power", [-60, -30, -22, 22, 30, 60])
def test_groups_of_very_different_size(d, group, power):
    """Values of one group of channels 2^power the size of the others': each group's weights keep their bits."""
    c = Call(5, [1, 3, 1], [1000, 70, 300], d, hk=2, share=3, group=group)
    factor = torch.ones(d // group, 1, dtype=torch.float64)
    factor[-1] = 2.0 ** power
    scaled(c, 1, factor)
    c.v[..., -group:] = (c.v[..., -group:].double() * 2.0 ** power).to(torch.bfloat16)
    c.dev[2].copy_(c.v)
    c.attend()
    assert not c.expanded
    c.check()


@pytest.mark.parametrize("d,group", DIMS)
@pytest.mark.parametrize("power", [60, 92])
def test_new_tokens_of_small_weight_beside_large_cached_values(d, group, power):
    """Cached keys outweigh the new tokens by 2^-14 to 2^-20 and hold 0 in every group's first channel, which is the new
    tokens' alone: their weights keep their bits under the factor of the cached ones'."""
    c = Call(8, [6, 1, 40], [300, 65, 32], d, hk=2, share=2, group=group)
    c.cache.codes[1][..., ::group // 2] &= 0xf0
    c.codes[1][1].copy_(c.cache.codes[1])
    c.cache.params[1][..., 1] = 0
    scaled(c, 1, 2.0 ** power)
    c.v = (c.v.double() * 2.0 ** power).to(torch.bfloat16)
    c.dev[2].copy_(c.v)
    c.q = c.q.abs()
    c.dev[0].copy_(c.q)
    up = 12 / (c.q.double().sum(-1).mean() * c.scale)
    c.cache.params[0][..., 1] = (c.cache.params[0][..., 1].double() + up).to(torch.bfloat16)
    c.params[0][1].copy_(c.cache.params[0])
    c.attend()
    assert not c.expanded
    c.check()


@pytest.mark.parametrize("d,group", [(128, 128), (128, 32), (32, 32)])
@pytest.mark.parametrize("new", [[1, 1], [1, 3]])
@pytest.mark.parametrize("power", [-90, -110, -118])
def test_tiny_values(d, group, new, power):
    """Cached values whose scales are near the smallest normal number."""
    c = Call(9, new, [500, 40], d, hk=2, share=3, group=group)
    scaled(c, 1, 2.0 ** power)
    c.v = (c.v.double() * 2.0 ** power).to(torch.bfloat16)
    c.dev[2].copy_(c.v)
    c.q *= 4
    c.dev[0].copy_(c.q)
    c.attend()
    assert not c.expanded
    c.check()


@pytest.mark.parametrize("d,group", [(128, 64), (128, 32), (64, 32)])
@pytest.mark.parametrize("power", [-40, -26, -22, -12])
@pytest.mark.parametrize("block", [0, 16])
def test_chunks_over_groups_of_very_different_size(d, group, power, block):
    """The tile kernel: values near 1 beside a group near 2^power, which keeps at least bf16's bits.  Queries are
    large: few keys weigh at all, so that errors do not cancel."""
    c = Call(6, [400, 1, 129], [700, 129, 128], d, hk=1, share=16, group=group, block=block)
    factor = torch.ones(d // group, 1, dtype=torch.float64)
    factor[-1] = 2.0 ** power
    scaled(c, 1, factor)
    c.v[..., -group:] = (c.v[..., -group:].double() * 2.0 ** power).to(torch.bfloat16)
    c.dev[2].copy_(c.v)
    c.q *= 4
    c.dev[0].copy_(c.q)
    c.attend()
    assert c.expanded
    c.check(tiles=True, halves=False)


@pytest.mark.parametrize("block", [0, 16])
def test_chunks_over_rows_of_very_different_size(block):
    """One position in 16 holds values near 2^-26 and scores highest."""
    c = Call(7, [400, 1, 129], [700, 129, 128], hk=1, share=16, group=32, block=block)
    rows = torch.arange(c.cache.codes[0].shape[2]) % 16 == 3
    scaled(c, 1, torch.where(rows, 2.0 ** -26, 1.0)[:, None, None].double())
    c.q = c.q.abs()
    c.dev[0].copy_(c.q)
    up = 30 / (c.q.double().sum(-1).mean() * c.scale)
    c.cache.params[0][..., 1] = (c.cache.params[0][..., 1].double() + up * rows[:, None]).to(torch.bfloat16)
    c.params[0][1].copy_(c.cache.params[0])
    c.attend()
    assert c.expanded
    c.check(tiles=True, halves=False)



@pytest.mark.parametrize("nats", [4, 10, 60])
def test_chunks_over_large_values_of_one_sign(nats):
    """Values near the largest allowed, all positive, under scores that rise over the maximum of the first tiles: by
    less than it may fall behind, and by more."""
    c = Call(10, [700], [9000], 32, hk=1, share=16, group=32)
    c.q = c.q.abs()
    c.dev[0].copy_(c.q)
    up = nats / (c.q.double().sum(-1).mean() * c.scale)
    later = torch.arange(c.cache.cap) >= 256
    c.cache.params[0][..., 1] = (c.cache.params[0][..., 1].double() + up * later[:, None]).to(torch.bfloat16)
    c.params[0][1].copy_(c.cache.params[0])
    c.cache.params[1][..., 1] = 0
    scaled(c, 1, 2.0 ** 76)
    c.v = (c.v.double().abs() * 2.0 ** 76).to(torch.bfloat16)
    c.dev[2].copy_(c.v)
    c.attend()
    assert c.expanded
    c.check(tiles=True, halves=False)


# ---------------------------------------------------------------------------
# which way sequences go
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens,fit", [
    ([131000, 131000, 1000, 0], [0, 2, 3]),
    ([131000, 50000, 131000, 40000, 5000, 3000, 0], [0, 3, 5, 6]),
    ([0, 131000, 0, 44000, 43000, 600, 500, 0], [0, 1, 2, 4, 5, 7]),  # 1365 - 1024 - 336 - 5 = 0 blocks for the 500
])
def test_what_fits_is_expanded_whatever_stands_before_it(lens, fit):
    """The 1 GiB of expanded blocks holds 1365 of 128 positions of 8 heads: sequences are taken in order as long as
    they fit in what is left, and a first prompt needs no room.  The tile kernel's bits for a sequence are the
    same whatever its neighbours; the row kernel's differ.  (Cached positions are 64 blocks over and over.)"""
    g = torch.Generator().manual_seed(18)
    hk, d, bs, n, seqs = 8, 128, 16, 400, len(lens)
    per, own = -(-(max(lens) + n) // bs), n // bs + 2
    cache = R.Cache(g, 1, (64 + 2 * seqs * own) * bs, hk, d, 128, bs, spare=0)
    codes, params = [x.cuda() for x in cache.codes], [x.cuda() for x in cache.params]
    q, k, v = ((torch.randn((seqs * n, hk, d), generator=g) * s).to(torch.bfloat16).cuda() for s in (3, 1, 1))
    short = [p if b in fit else 0 for b, p in enumerate(lens)]  # (which needs no room)
    table = torch.randint(0, 64, (seqs, per), generator=g)
    for b in range(seqs):                        # blocks of its own for what a call writes
        for i, p in enumerate((short[b], lens[b])):
            at = torch.arange(p // bs, min(p // bs + own, per))
            table[b, at] = 64 + (2 * b + i) * own + torch.arange(len(at))
    i32 = dict(dtype=torch.int32, device="cuda")
    table = table.to(**i32)

    def attend(lens):
        cu, cu_k = [0], [0]
        for p in lens:
            cu.append(cu[-1] + n)
            cu_k.append(cu_k[-1] + n + p)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        c = [x.clone() for x in codes + params]
        binding.prefill_attn_varlen_cache4(q, k, v, torch.tensor(cu, **i32), torch.tensor(cu_k, **i32), c[0], c[1],
                                           torch.tensor(lens, **i32), out, lse, cache_k_params=c[2], cache_v_params=c[3],
                                           block_table=table)
        assert binding.load().prefill_attn_last_schedule() != 0
        torch.cuda.synchronize()
        assert binding.prefill_attn_device_status() == 0
        return out, lse

    crowded, roomy = attend(lens), attend(short)
    for got, want in zip(crowded, roomy):
        assert got.isfinite().all()
        for b in fit:
            assert torch.equal(got[b * n:(b + 1) * n], want[b * n:(b + 1) * n]), b


# ---------------------------------------------------------------------------
# copies
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("block", [0, 8])
def test_copies_of_many_sequences(block):
    """More sequences than a block searches in shared memory, empty ones among them."""
    g = torch.Generator().manual_seed(19)
    new = torch.randint(0, 3, (1500,), generator=g).tolist()
    lens = torch.randint(0, 20, (1500,), generator=g).tolist()
    c = Call(20, new, lens, 32, hk=2, group=32, block=block)
    c.write()
    k, v = torch.empty_like(c.dev[1]), torch.empty_like(c.dev[2])
    binding.prefill_attn_cache4_read(c.codes[0][1], c.codes[1][1], c.meta[0], c.offsets, k, v, **c.opts)
    torch.cuda.synchronize()
    assert binding.prefill_attn_device_status() == 0
    c.check_cache()
    c.guards()
    for got, x in ((k, c.k), (v, c.v)):
        assert same_bits(got, R.values(*R.quantise(x, 32)).float().to(torch.bfloat16))


def test_captured_copies_read_their_metadata_at_replay():
    c = Call(21, [40, 0, 90, 3], [7, 0, 64, 1], group=64, block=16)
    k, v = torch.empty_like(c.dev[1]), torch.empty_like(c.dev[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def copies():
        c.write()
        binding.prefill_attn_cache4_read(c.codes[0][1], c.codes[1][1], c.meta[0], c.offsets, k, v, **c.opts)

    with torch.cuda.stream(side):
        copies()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            copies()
        d = Call(22, [1, 90, 2, 40], [100, 0, 31, 64], group=64, block=16, slack=154 + 3 - 104)
        for a, b in zip(c.codes + c.params, d.codes + d.params):
            a[1].copy_(b[1])
        for a, b in zip([*c.dev, *c.meta, c.offsets, c.opts["block_table"]],
                        [*d.dev, *d.meta, d.offsets, d.opts["block_table"]]):
            a.copy_(b)
        graph.replay()
    side.synchronize()
    d.codes, d.params = c.codes, c.params
    d.check_cache()
    for got, x in ((k, d.k), (v, d.v)):
        assert same_bits(got, R.values(*R.quantise(x, 64)).float().to(torch.bfloat16))
