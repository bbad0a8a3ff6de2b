"""Paged-cache operators where their inputs are malformed or at the edge of a type: what the
device must notice, and what must not leak into the rows beside it."""
import pytest
import torch

from masked_discrete_diffusion_b200 import binding, build
from test_gpu_paged import BF16, F16, Pages, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def guarded(rows, *shape, dt):
    """A tensor of sevens and its middle `rows` rows."""
    mem = torch.full((rows + 16, *shape), 7.0, dtype=dt, device="cuda")
    return mem, mem[8:8 + rows]


# ------------------------------------------------------------------ decreasing q_start
@pytest.mark.parametrize("B,n", [(4, 40), (3, 300), (500, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_skips_a_batch_whose_chunks_overlap(B, n, causal):
    """q_start = 0, n, 0, n, ..: every second sequence is in order by itself and has all rows.
    Nothing is written, inside out and lse or beside them, and the next call is right."""
    pg = Pages([(n, 400)] + [(0, 400)] * (B - 1), 2, 64, 64, BF16)
    q = rnd(1, n, 8, 64)
    want = binding.dg_paged_attention(pg.cache, pg.batch, q, causal)
    good = pg.q_start.clone()
    for bad in ([n * (i % 2) for i in range(B + 1)], [0] + [n] * (B - 1) + [n - 1]):
        pg.q_start.copy_(torch.tensor(bad, dtype=torch.int32))
        mem, out = guarded(n, 8, 64, dt=BF16)
        lmem, lse = guarded(n, 8, dt=torch.float32)
        err = err_word()
        binding.dg_paged_attention(pg.cache, pg.batch, q, causal, out=out, lse=lse, err=err)
        assert int(err) == binding.PAGED_BAD_BATCH
        assert bool((mem == 7).all()) and bool((lmem == 7).all())
    pg.q_start.copy_(good)
    err = err_word()
    assert torch.equal(binding.dg_paged_attention(pg.cache, pg.batch, q, causal, err=err), want)
    binding.dg_paged_check(err)


def test_attention_skips_overlapping_chunks_whose_tiles_pass_32_bits():
    """The same with chunks and tables so long that the accepted sequences' key tiles would
    number more than 2^31 together, while the rows counted once stay below."""
    n, hq, hkv, h, ps = 262144, 128, 8, 64, 1024
    k = rnd(2, 1, ps, hkv, h, dt=F16)
    cache = binding.PagedCache(k, k.clone())
    table = torch.zeros(4, 1024, dtype=torch.int32, device="cuda")
    kv = torch.full((4,), 1 << 20, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n, 0, n, 0], dtype=torch.int32, device="cuda")
    batch = binding.PagedBatch(start, kv, table, n)
    q = torch.zeros(n, hq, h, dtype=F16, device="cuda")
    out = torch.full((n, hq, h), 7.0, dtype=F16, device="cuda")
    err = err_word()
    binding.dg_paged_attention(cache, batch, q, False, out=out, err=err)
    assert int(err) == binding.PAGED_BAD_BATCH
    assert all(bool((x == 7).all()) for x in out.split(1 << 15))


# ------------------------------------------------------------------ bad pages
@pytest.mark.parametrize("dt,h", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_bad_pages_of_single_tile_sequences_make_whole_rows_nan(dt, h, causal):
    """Sequences of one key tile, more of them than a CTA's flags have places for: all channels
    of a sequence with a bad page are NaN, and no other row changes a bit."""
    shapes = [(1, 40), (1, 128), (2, 20), (20, 100), (1, 1), (3, 77)]
    pg = Pages([shapes[i % 6] for i in range(600)], 4, h, 16, dt)
    q = rnd(31, pg.n, 8, h, dt=dt)
    clean = binding.dg_paged_attention(pg.cache, pg.batch, q, causal)
    assert torch.isfinite(clean).all()
    rotten = torch.zeros(pg.n, dtype=torch.bool, device="cuda")
    for b in range(0, 600, 7):
        pg.table[b, 0] = -1 if b % 2 else pg.k.shape[0]
        rotten[pg.starts[b]:pg.starts[b + 1]] = True
    for _ in range(20):
        err, lse = err_word(), torch.zeros(pg.n, 8, device="cuda")
        got = binding.dg_paged_attention(pg.cache, pg.batch, q, causal, lse=lse, err=err)
        assert int(err) == binding.PAGED_BAD_PAGE
        assert bool(got[rotten].isnan().all()) and bool(lse[rotten].isnan().all())
        assert torch.equal(got[~rotten], clean[~rotten])


# ------------------------------------------------------------------ small weights
@pytest.mark.parametrize("dt", [BF16, F16])
@pytest.mark.parametrize("h,seqs,causal", [(64, [(1, 65537), (1, 3000)], True),
                                           (128, [(130, 20000)], False), (64, [(3, 129)], True)])
@pytest.mark.parametrize("below", [14.25, 18.375, 21.5, 24.5, 27.25])
def test_many_small_weights_beside_a_large_one(dt, h, seqs, causal, below):
    """One key (an attention sink, its value 0) whose weight is 2^below times that of every
    other key, whose values are 1.  The scores are sums of two products of few bits, so their
    fp32 sums are exact; `below` is taken in units of log 2 by the scale.

    The result is n 2^-below / (1 + n 2^-below) for n other keys.  Off by: half a step of each
    weight and of the result (2 u of it); f16's steps, the largest weight standing at 2^7: at
    most 2^-32 of the largest weight a key, n 2^-32 / (1 + n 2^-below) in all; the result's
    subnormal step (2^-25 in f16); fp32's share as in the attention test, (384 + n / 64) 2^-23
    of the result; 2^-20 for exp2 and the exponent's rounding (below 2^5: 2^-20 of a power); and
    the scale, which is 1 / log2(e) to within three roundings: `below` 3 2^-24 of a power."""
    hq, hkv, ps = 4, 2, 64
    pg = Pages(seqs, hkv, h, ps, dt)
    pg.k.zero_(), pg.v.fill_(1)
    q = torch.zeros(pg.n, hq, h, dtype=dt, device="cuda")
    q[..., 0] = 1
    for b in range(len(seqs)):
        page, slot = pg.slots(b, 5, 6)
        pg.k[page, slot, :, 0] = below
        pg.v[page, slot] = 0
    scale = 0.6931471805599453
    got = binding.dg_paged_attention(pg.cache, pg.batch, q, causal, scale=scale).double()
    u = torch.finfo(dt).eps / 2
    for b, (ql, kv) in enumerate(seqs):
        rows = got[pg.starts[b]:pg.starts[b + 1]]
        n = torch.tensor([(kv - ql + i + 1 if causal else kv) - 1 for i in range(ql)],
                         dtype=torch.float64, device="cuda")[:, None, None]
        mass = n * 2.0 ** -below
        want = mass / (1 + mass)
        tol = 2 * u * want + ((384 + n / 64) * 2.0 ** -23 + 2.0 ** -20
                                + below * 3 * 2.0 ** -24) * want
        if dt == F16:
            tol = tol + n * 2.0 ** -32 / (1 + mass) + 2.0 ** -25
        assert float(((rows - want).abs() - tol).max()) <= 0


# ------------------------------------------------------------------ append's checks
@pytest.mark.parametrize("starts,lens", [
    ([0, 10, 5, 20], [20, 20, 20]),                  # decreasing, every chunk within max_q
    ([0, 20, 20, 20], [20, -1, 20]),                 # an empty chunk with a negative length,
    ([0, 20, 20, 20], [20, 20, 33]),                 # with one that its table cannot hold
    ([0, 0, 0, 21], [0, 0, 21]),                     # rows that the call does not have
    ([-5, -2, 0, 20], [20, 20, 20]),                 # chunks in front of the rows
    ([0] * 100 + [7, 20] + [20] * 50, [20] * 120 + [40] + [20] * 30),
], ids=str)
def test_append_and_attention_flag_the_same_batches(starts, lens):
    """Every fault of the batch sets the bit, whether or not a row meets it."""
    B = len(lens)
    assert len(starts) == B + 1
    pages = rnd(41, 2 * B, 16, 2, 64)
    cache = binding.PagedCache(pages, pages.clone())
    table = torch.arange(2 * B, device="cuda", dtype=torch.int32).view(B, 2)
    x = rnd(42, 20, 2, 64)

    def bits(starts, lens):
        batch = binding.PagedBatch(torch.tensor(starts, dtype=torch.int32, device="cuda"),
                                   torch.tensor(lens, dtype=torch.int32, device="cuda"), table, 20)
        a, b = err_word(), err_word()
        binding.dg_paged_append(cache, batch, x, x, err=a)
        binding.dg_paged_attention(cache, batch, x, err=b)
        return int(a), int(b)

    assert bits(starts, lens) == (binding.PAGED_BAD_BATCH, binding.PAGED_BAD_BATCH)
    assert bits([0] * B + [20], [20] * B) == (0, 0)


def test_chunks_beyond_a_bound_of_no_rows_are_flagged():
    """max_q = 0: any chunk is too long for both operators; a batch of empty chunks is fine."""
    pg = Pages([(2, 600), (0, 20)], 2, 64, 16, BF16)
    batch = binding.PagedBatch(pg.q_start, pg.kv_len, pg.table, 0)
    q, kv = rnd(51, 2, 4, 64), rnd(52, 2, 2, 64)
    for want in (binding.PAGED_BAD_BATCH, 0):
        mem, out = guarded(2, 4, 64, dt=BF16)
        keep = pg.kmem.clone()
        a, b = err_word(), err_word()
        binding.dg_paged_append(pg.cache, batch, kv, kv, err=a)
        binding.dg_paged_attention(pg.cache, batch, q, out=out, err=b)
        binding.dg_paged_attention(pg.cache, batch, q, out=out)
        assert (int(a), int(b)) == (want, want)
        assert bool((mem == 7).all()) and torch.equal(pg.kmem, keep)
        pg.q_start.zero_()


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("dt,h,seqs,causal", [
    (BF16, 128, [(1, 40)], True), (BF16, 128, [(1, 5000), (9, 9000)], True),
    (F16, 64, [(300, 700), (1, 1000), (130, 130)], False), (BF16, 64, [(1, 90)] * 700, True)])
def test_a_wait_that_runs_out_is_reported_and_leaves_the_operator_usable(dt, h, seqs, causal):
    """The values never come (the launch does not load them): the call ends by itself, says so,
    and the calls after it have the bits of those before."""
    pg = Pages(seqs, 2, h, 16, dt)
    q = rnd(71, pg.n, 8, h, dt=dt)
    want = binding.dg_paged_attention(pg.cache, pg.batch, q, causal)
    for _ in range(2):
        err = err_word()
        binding.dg_debug_stall_paged(5_000_000)  # 5 ms a wait
        binding.dg_paged_attention(pg.cache, pg.batch, q, causal, err=err)
        with pytest.raises(binding.DGError, match="wait") as e:
            binding.dg_paged_check(err)
        assert e.value.status == 5 and int(err) == binding.PAGED_TIMEOUT
        for _ in range(3):
            err = err_word()
            assert torch.equal(binding.dg_paged_attention(pg.cache, pg.batch, q, causal, err=err),
                               want)
            binding.dg_paged_check(err)


# ------------------------------------------------------------------ the cache's own error word
def test_calls_without_an_err_report_to_their_cache():
    pg, other = (Pages([(2, 40), (3, 20)], 2, 64, 16, BF16) for _ in range(2))
    q, kv = rnd(81, 5, 4, 64), rnd(82, 5, 2, 64)

    def both(p, err=None):
        binding.dg_paged_append(p.cache, p.batch, kv, kv, err=err)
        return binding.dg_paged_attention(p.cache, p.batch, q, err=err)

    both(pg)
    binding.dg_paged_check(pg.cache)
    pg.table[1, 0] = -1
    both(pg), both(other)
    with pytest.raises(binding.DGError, match="page number"):
        binding.dg_paged_check(pg.cache)
    binding.dg_paged_check(pg.cache)     # the report has cleared it
    binding.dg_paged_check(other.cache)  # and the other cache never saw it
    mine = err_word()
    both(pg, mine)
    assert int(mine) == binding.PAGED_BAD_PAGE
    binding.dg_paged_check(pg.cache)     # a caller's word is used instead
    pg.kv_len[0] = 1000
    binding.dg_paged_append(pg.cache, pg.batch, kv, kv)
    with pytest.raises(binding.DGError, match="kv_len"):
        binding.dg_paged_check(pg.cache)
    # captured: every replay reports
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both(pg)
    binding.dg_paged_check(pg.cache)
    for _ in range(2):
        graph.replay()
        with pytest.raises(binding.DGError, match="kv_len"):
            binding.dg_paged_check(pg.cache)
