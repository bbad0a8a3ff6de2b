"""The paged-cache operators against plain fp64 implementations.

Tolerances, with u = eps/2 of the type (half a step) and f = 2^-24 (fp32's):

* norm and rotation: one rounding to the type (u of the result), and in fp32 at most 26
  roundings to the root (16 squares a lane, 4 adds across lanes, quotient, sum, root,
  reciprocal), 2 for the gain, 3 for the rotation, and sines of an angle cut to 2^-25 half
  turns and computed to 2 units of fp32 (pi f + 2 f of their arguments' pair); together
  under 48 f of |a| + |b| for a pair (a, b).
* attention: the weights are rounded to the type (u of sum p|v|) and so is the result (u of
  it); scores are sums of h products in fp32, off by (h + 4) f of the largest sum of
  |q k| scale, S, which changes each weight by twice that, exp2 by under 4 f of itself more.
  The fp32 sum over n keys (blocks of at most 128 added in a chain, each block's values one
  by one, at most 2^8 rescalings and as many pieces) rounds at most 128 + n / 64 + 256
  times, in the numerator and in the denominator.  (A piece is added after at most 148
  others, a tile holds two additions to the chain, and a row whose maximum moves in more
  than 2^8 tiles has lost the earlier ones to 2^-2048.)
"""
import math

import numpy as np
import pytest
import torch

from masked_discrete_diffusion_b200 import binding, build

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
F = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def rnd(seed, *shape, dt=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dt)


# ------------------------------------------------------------------ norm and rotation
def turned(x, gain, eps, pos, base):
    """(value, bound) in fp64 of the norm and rotation of x [n, heads, h]."""
    y = x.double()
    h = y.shape[-1]
    if eps is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt()
        if gain is not None:
            y = y * gain.double()
    a, b = y[..., :h // 2], y[..., h // 2:]
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    bound = 48 * F * size
    if base is not None:
        inv = base ** (-torch.arange(0, h, 2, device="cuda", dtype=torch.float64) / h)
        ang = (pos.double()[:, None] * inv)[:, None, :]
        # this reference's own angle: a few fp64 roundings of the angle itself
        bound = bound + (2.0 ** -50 * ang.abs()).repeat(1, 1, 2) * size
        y = torch.cat((a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()), -1)
    return y, bound + half_step(x.dtype) * y.abs() + 1e-30


def tiny(dt):
    """Half the smallest step of f16's subnormals; nothing for the wider exponents."""
    return 2.0 ** -25 if dt == F16 else 0.0


def check(got, want, bound, dt=None):
    over = (got.double() - want).abs() - bound - (tiny(dt) if dt else 0)
    assert torch.isfinite(got).all() and float(over.max()) <= 0, float(over.max())


NORM = [  # dtype, n, hq, hkv, h, gains, eps, base, far
    (BF16, 1, 16, 8, 128, True, 1e-6, 1e4, 1024),
    (BF16, 257, 16, 8, 128, True, 1e-6, 1e4, 1 << 20),
    (F16, 1000, 12, 4, 64, True, 1e-5, 5e5, 1 << 30),
    (F32, 333, 4, 2, 16, False, 1e-6, 1e4, 4096),
    (F32, 3, 7, 1, 256, True, 1e-6, 1e6, 1 << 20),
    (BF16, 64, 3, 3, 96, True, 0.0, 1e4, 100),
    (F16, 5, 1, 1, 80, False, None, 1e4, 100),
    (BF16, 6000, 71, 1, 64, True, 1e-6, None, 1),
    (F32, 20000, 16, 8, 128, True, 1e-6, 1e4, 1 << 17),
    (BF16, 9, 2, 1, 48, False, 1e-6, 1.0, 7),
]


@pytest.mark.parametrize("case", NORM, ids=str)
def test_norm_rope_matches_fp64(case):
    dt, n, hq, hkv, h, gains, eps, base, far = case
    q, k = rnd(1, n, hq, h, dt=dt), rnd(2, n, hkv, h, dt=dt) * 3
    qg = rnd(3, h, dt=dt) if gains else None
    kg = rnd(4, h, dt=dt) if gains else None
    pos = torch.randint(-far, far, (n,), device="cuda", dtype=torch.int32)
    rope = binding.dg_rope_init(base, h) if base else None
    qo, ko = binding.dg_qk_norm_rope(q, k, pos, rope, qg, kg, eps)
    check(qo, *turned(q, qg, eps, pos, base), dt)
    check(ko, *turned(k, kg, eps, pos, base), dt)


def test_norm_rope_in_place_on_strided_rows():
    """Views of a QKV projection's rows, heads-first views, and in place: the same bits."""
    n, hq, hkv, h = 100, 6, 2, 64
    x = rnd(5, n, hq + 2 * hkv, h)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    rope = binding.dg_rope_init(1e4, h)
    q, k = x[:, :hq], x[:, hq:hq + hkv]
    a = binding.dg_qk_norm_rope(q.contiguous(), k.contiguous(), pos, rope)
    t = torch.empty(hq, n, h, dtype=BF16, device="cuda")
    b = binding.dg_qk_norm_rope(q, k, pos, rope, q_out=t.transpose(0, 1))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    rest = x[:, hq + hkv:].clone()
    binding.dg_qk_norm_rope(q, k, pos, rope, q_out=q, k_out=k)
    assert torch.equal(a[0], q) and torch.equal(a[1], k) and torch.equal(rest, x[:, hq + hkv:])


def test_norm_rope_empty_and_single_sided():
    z = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    qo, ko = binding.dg_qk_norm_rope(z, z, torch.empty(0, dtype=torch.int32, device="cuda"),
                                     binding.dg_rope_init(1e4, 64))
    assert qo.shape == z.shape and ko.shape == z.shape
    q, none = rnd(6, 5, 4, 64), torch.empty(5, 0, 64, dtype=BF16, device="cuda")
    qo, ko = binding.dg_qk_norm_rope(q, none)
    check(qo, *turned(q, None, 1e-6, None, None), BF16)
    zero = torch.zeros(2, 1, 64, dtype=BF16, device="cuda")
    assert torch.equal(binding.dg_qk_norm_rope(zero, zero)[0], zero)


# ------------------------------------------------------------------ pages
class Pages:
    """A pool of pages in one of four memory orders, a table of shuffled pages, and the
    batch of sequences (chunk length, length with the chunk)."""

    def __init__(self, seqs, hkv, h, ps, dt, order="page", pad=0, fill=None, seed=0, extra=2,
                 lead=0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.ps, self.pad, self.lead = seqs, ps, pad, lead
        need = [-(-kv // ps) for _, kv in seqs]
        n = sum(need) + extra
        shape = {"page": (n, ps, hkv, h), "head": (n, hkv, ps, h), "heads_first": (hkv, n, ps, h),
                 "wide": (n, ps, hkv + 1, h)}[order]
        view = {"page": lambda x: x, "head": lambda x: x.transpose(1, 2),
                "heads_first": lambda x: x.permute(1, 2, 0, 3), "wide": lambda x: x[:, :, :hkv]}
        make = (lambda s: rnd(seed + s, *shape, dt=dt)) if fill is None else (
            lambda s: torch.full(shape, fill, dtype=dt, device="cuda"))
        self.kmem, self.vmem = make(1), make(2)
        self.k, self.v = view[order](self.kmem), view[order](self.vmem)
        perm = torch.randperm(n, generator=g).tolist()
        table = torch.full((len(seqs), max(need + [1])), -1, dtype=torch.int32)
        for b, m in enumerate(need):
            for i in range(m):
                table[b, i] = perm.pop()
        self.table = table.cuda()
        starts = [lead]
        for q, _ in seqs:
            starts.append(starts[-1] + q)
        self.starts, self.n = starts, starts[-1] + pad
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([kv for _, kv in seqs], dtype=torch.int32, device="cuda")
        self.max_q = max([q for q, _ in seqs] + [0])
        self.cache = binding.PagedCache(self.k, self.v)
        self.batch = binding.PagedBatch(self.q_start, self.kv_len, self.table, self.max_q)

    def slots(self, b, lo, hi):
        p = torch.arange(lo, hi, device="cuda")
        return self.table[b].long()[p // self.ps], p % self.ps


APPEND = [  # dtype, hq, hkv, h, page, order, seqs (chunk, total), pad
    (BF16, 16, 8, 128, 16, "page", [(1, 1), (1, 33), (1, 16), (1, 17)], 0),
    (F16, 12, 4, 64, 32, "head", [(5, 37), (0, 50), (64, 64), (1, 32)], 3),
    (BF16, 0, 1, 96, 64, "heads_first", [(200, 700), (129, 129)], 0),
    (F16, 2, 2, 16, 128, "wide", [(7, 9), (300, 1000), (0, 0)], 11),
    (BF16, 7, 1, 256, 16, "page", [(i % 4, 3 * i + 4) for i in range(70)], 0),
    (BF16, 4, 2, 64, 16, "page", [(9, 4), (3, 3)], 0),  # rows before position 0
]


@pytest.mark.parametrize("case", APPEND, ids=str)
def test_append_matches_fp64(case):
    dt, hq, hkv, h, ps, order, seqs, pad = case
    pg = Pages(seqs, hkv, h, ps, dt, order, pad, lead=2)
    x = rnd(9, pg.n, hq + 2 * hkv, h, dt=dt)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    qg, kg = rnd(10, h, dt=dt), rnd(11, h, dt=dt)
    rope = binding.dg_rope_init(1e4, h)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw, vw = pg.k.double(), pg.v.double()
    kb, vb = torch.zeros_like(kw), torch.zeros_like(vw)
    out = torch.full((pg.n, hq, h), 7.0, dtype=dt, device="cuda")
    qw, qb = out.double(), torch.zeros(pg.n, hq, h, dtype=torch.float64, device="cuda")
    for b, (ql, kv) in enumerate(seqs):
        lo, hi = pg.starts[b], pg.starts[b + 1]
        pos = torch.arange(kv - ql, kv, device="cuda")
        w, bd = turned(k[lo:hi], kg, 1e-6, pos, 1e4)
        cut = max(0, ql - kv)
        page, slot = pg.slots(b, max(0, kv - ql), kv)
        kw[page, slot], kb[page, slot] = w[cut:], bd[cut:]
        vw[page, slot] = v[lo + cut:hi].double()
        if hq:
            qw[lo:hi], qb[lo:hi] = turned(q[lo:hi], qg, 1e-6, pos, 1e4)
    edge = pg.kmem.clone()
    res = binding.dg_paged_append(pg.cache, pg.batch, k, v, rope, kg, 1e-6,
                                  q if hq else None, qg if hq else None, out if hq else None, err)
    assert (res is out) if hq else res is None
    binding.dg_paged_check(err)
    check(pg.k, kw, kb, dt)
    assert torch.equal(pg.v.double(), vw)
    if hq:
        check(out, qw, qb, dt)
    if order == "wide":  # memory beside the cache's heads is left alone
        assert torch.equal(pg.kmem[:, :, hkv], edge[:, :, hkv])
    # as they are, without norm or rotation
    binding.dg_paged_append(pg.cache, pg.batch, k, v)
    for b, (ql, kv) in enumerate(seqs):
        cut, page_slot = max(0, ql - kv), pg.slots(b, max(0, kv - ql), kv)
        assert torch.equal(pg.k[page_slot], k[pg.starts[b] + cut:pg.starts[b + 1]])


def test_append_skips_bad_pages_and_lengths():
    pg = Pages([(2, 40), (3, 20), (2, 18), (4, 4)], 2, 64, 16, BF16)
    k, v = rnd(1, pg.n, 2, 64), rnd(2, pg.n, 2, 64)
    good_k, good_v = pg.k.clone(), pg.v.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pg.table[0, 2] = pg.k.shape[0]      # both new rows of sequence 0
    pg.table[1, 1] = -5                 # all three of sequence 1
    pg.kv_len[3] = pg.table.shape[1] * 16 + 1
    binding.dg_paged_append(pg.cache, pg.batch, k, v, err=err)
    with pytest.raises(binding.DGError, match="page number"):
        binding.dg_paged_check(err)
    assert int(err) == binding.PAGED_BAD_BATCH | binding.PAGED_BAD_PAGE
    s = pg.slots(2, 16, 18)
    good_k[s], good_v[s] = k[5:7], v[5:7]
    assert torch.equal(pg.k, good_k) and torch.equal(pg.v, good_v)
    # chunk bounds outside the rows, decreasing, or longer than max_q: skipped as well
    for bad in ([0, 2, 5, 7, 12], [-1, 2, 5, 7, 11], [0, 5, 2, 7, 11]):
        err.zero_()
        pg.kv_len.fill_(20)
        pg.table.copy_(Pages([(2, 40), (3, 20), (2, 18), (4, 4)], 2, 64, 16, BF16).table)
        pg.q_start.copy_(torch.tensor(bad, dtype=torch.int32))
        binding.dg_paged_append(pg.cache, pg.batch, k, v, err=err)
        assert int(err) & binding.PAGED_BAD_BATCH


# ------------------------------------------------------------------ attention
def seen_range(ql, kv, causal, window, i):
    past = kv - ql
    hi = min(kv, past + i + 1) if causal else kv
    lo = max(0, (past + i + 1 if causal else past) - window) if window else 0
    return lo, hi


def attention_fp64(pg, q, flags, window, scale):
    """(out, bound, lse, lse bound) of every row of every sequence."""
    n, hq, h = q.shape
    hkv = pg.k.shape[2]
    u = half_step(q.dtype)
    out = torch.zeros(n, hq, h, dtype=torch.float64, device="cuda")
    bound, lse = torch.zeros_like(out), torch.full((n, hq), -math.inf, dtype=torch.float64,
                                                  device="cuda")
    lbound = torch.zeros_like(lse)
    for b, (ql, kv) in enumerate(pg.seqs):
        if not ql:
            continue
        page, slot = pg.slots(b, 0, kv)
        rng = [seen_range(ql, kv, flags[b], window, i) for i in range(ql)]
        lo = torch.tensor([r[0] for r in rng], device="cuda")[:, None]
        hi = torch.tensor([r[1] for r in rng], device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None]
        vis = (j >= lo) & (j < hi)
        used = vis.any(0)
        for g in range(hkv):
            kk, vv = pg.k[page, slot, g].double(), pg.v[page, slot, g].double()
            kk, vv = kk.masked_fill(~used[:, None], 0), vv.masked_fill(~used[:, None], 0)
            for r in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                rows = slice(pg.starts[b], pg.starts[b + 1])
                qq = q[rows, r].double()
                x = (qq @ kk.T * scale).masked_fill(~vis, -math.inf)
                S = (qq.abs() @ kk.abs().T * scale).masked_fill(~vis, 0)
                m = x.amax(-1, keepdim=True) if kv else None
                if not kv:
                    continue
                e = torch.where(vis, (x - m.clamp(min=-1e300)).exp(), torch.zeros_like(x))
                den = e.sum(-1, keepdim=True)
                p = e / den.clamp(min=1e-300)
                out[rows, r] = p @ vv
                pv = p @ vv.abs()
                grow = 2 * (h + 4) * F * S.amax(-1, keepdim=True) + 8 * F
                grow = grow + 2 * (384 + kv / 64) * F
                bound[rows, r] = (u + grow) * pv + u * out[rows, r].abs()
                live = vis.any(-1)
                lse[rows, r] = torch.where(live, m[:, 0] + den[:, 0].clamp(min=1e-300).log(),
                                           lse[rows, r])
                # the log of a sum off by `grow` of itself, and fp32's step at the value
                lbound[rows, r] = grow[:, 0] + 4 * F * (1 + lse[rows, r].abs().nan_to_num(posinf=0))
    return out, bound, lse, lbound


B, C = False, True
ATTEND = [  # dtype, h, hq, hkv, page, order, [(chunk, total)], causal flags, window
    (BF16, 128, 16, 8, 64, "page", [(1, 1024)], C, 0),
    (BF16, 128, 16, 8, 16, "page", [(1, 1), (1, 2), (1, 127), (1, 128), (1, 129)], C, 0),
    (F16, 64, 8, 8, 16, "head", [(1, 1000), (2, 17), (1, 15)], C, 0),
    (BF16, 128, 16, 8, 64, "page", [(256, 1280), (256, 256)], B, 1024),
    (BF16, 128, 16, 8, 64, "head", [(256, 2000), (96, 400), (256, 300)], B, 256),
    (F16, 64, 4, 2, 128, "heads_first", [(300, 300)], C, 0),
    (BF16, 64, 14, 2, 32, "page", [(77, 333), (129, 129), (1, 500), (0, 40)], C, 100),
    (F16, 128, 9, 3, 256, "wide", [(130, 700), (257, 257)], C, 1),
    (BF16, 128, 128, 1, 16, "page", [(3, 200), (1, 77)], C, 0),
    (F16, 128, 5, 1, 32, "page", [(40, 40), (25, 26), (26, 1000), (51, 51), (52, 60)], C, 0),
    (BF16, 64, 2, 2, 1024, "page", [(700, 1500)], "mixed", 300),
    (BF16, 128, 16, 8, 64, "page", [(256, 900), (256, 1800), (256, 256), (100, 640)], "mixed", 0),
    (BF16, 128, 4, 4, 16, "page", [(9, 4), (3, 0), (5, 5)], C, 0),      # rows that see nothing
    (F16, 64, 4, 4, 16, "page", [(9, 4), (3, 0), (5, 5)], B, 2),
    (BF16, 128, 32, 4, 32, "page", [(9, 9000), (4, 5001), (1, 12000)], C, 0),
    (BF16, 128, 8, 1, 16, "page", [(1, 40 + 61 * i) for i in range(150)], C, 0),
    (F16, 64, 12, 4, 32, "page", [(i % 5, 40 + 7 * i) for i in range(40)], "mixed", 33),
    (BF16, 128, 2, 1, 128, "page", [(1500, 1500)], C, 0),
    (BF16, 128, 2, 2, 128, "page", [(1, 100000)], C, 0),
    (F16, 64, 2, 1, 16, "page", [(300, 100), (257, 0), (200, 201)], C, 0),  # long dead stretches
    (BF16, 128, 128, 1, 64, "page", [(70, 200), (3, 9)], C, 40),        # items of two tokens
    (F16, 64, 4, 1, 16, "page", [(1, 1 + i % 70) for i in range(900)], C, 0),
    (BF16, 64, 6, 2, 16, "page", [(1 + i % 3, 20 + i) for i in range(500)], "mixed", 37),
    (BF16, 128, 4, 2, 64, "page", [(700, 900), (1, 3000), (60, 61), (130, 2000)], "mixed", 0),
]


def flags_of(mode, n):
    return [i % 2 == 0 for i in range(n)] if mode == "mixed" else [bool(mode)] * n


def causal_arg(mode, flags):
    return torch.tensor(flags, dtype=torch.uint8, device="cuda") if mode == "mixed" else mode


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
@pytest.mark.parametrize("sharp", [1.0, 6.0])
def test_attention_matches_fp64(case, sharp):
    """sharp: the queries' scale; large scores make the running maximum move."""
    dt, h, hq, hkv, ps, order, seqs, mode, window = case
    pg = Pages(seqs, hkv, h, ps, dt, order, pad=3, lead=1)
    q = (rnd(21, pg.n, hq + 2, h) * sharp).to(dt)[:, 1:hq + 1]
    flags = flags_of(mode, len(seqs))
    want, bound, lse, lbound = attention_fp64(pg, q, flags, window, h ** -0.5)
    out = torch.full((pg.n, hq, h), 7.0, dtype=dt, device="cuda")
    got_lse = torch.full((pg.n, hq), 7.0, dtype=F32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.dg_paged_attention(pg.cache, pg.batch, q, causal_arg(mode, flags), window, out=out,
                               lse=got_lse, err=err)
    binding.dg_paged_check(err)
    rows = slice(pg.starts[0], pg.starts[-1])
    assert bool((out[:rows.start] == 7).all()) and bool((out[rows.stop:] == 7).all())
    assert bool((got_lse[:rows.start] == 7).all()) and bool((got_lse[rows.stop:] == 7).all())
    check(out[rows], want[rows], bound[rows], dt)
    dead = torch.isinf(lse[rows])
    assert torch.equal(torch.isneginf(got_lse[rows]), dead)
    off = (got_lse[rows].double() - lse[rows]).abs()[~dead] - lbound[rows][~dead]
    assert off.numel() == 0 or float(off.max()) <= 0, float(off.max())
    assert torch.equal(out[rows][dead], torch.zeros_like(out[rows][dead]))
    again = binding.dg_paged_attention(pg.cache, pg.batch, q, causal_arg(mode, flags), window)
    assert torch.equal(again[rows], out[rows])  # and without the optional outputs


@pytest.mark.parametrize("step", [0.02, 0.5, 3.0])
@pytest.mark.parametrize("seqs,causal", [([(1, 3000)], C), ([(200, 1000), (130, 700)], C),
                                         ([(96, 900)], B)], ids=str)
def test_attention_when_every_tile_raises_the_maximum(seqs, causal, step):
    """Scores that climb by `step` a position (in units of log e, up to 9,000 in all): the
    reference moves in every tile, in both halves of it, and old weights fade to nothing."""
    h, hq, hkv = 64, 4, 2
    pg = Pages(seqs, hkv, h, 16, BF16)
    q = rnd(61, pg.n, hq, h)
    q[..., 0] = 8.0  # sqrt(h): scale q.k gains k[..., 0]
    for b, (_, kv) in enumerate(seqs):
        page, slot = pg.slots(b, 0, kv)
        ramp = torch.arange(kv, device="cuda").float() * step
        pg.k[page, slot, :, 0] = ramp.to(BF16)[:, None]
    want, bound, _, _ = attention_fp64(pg, q, [causal] * len(seqs), 0, h ** -0.5)
    got = binding.dg_paged_attention(pg.cache, pg.batch, q, causal)
    check(got, want, bound, BF16)


@pytest.mark.parametrize("rot", [float("nan"), float("inf")])
@pytest.mark.parametrize("case", [ATTEND[i] for i in (1, 3, 6, 9, 12, 13, 16)],
                         ids=lambda c: str(c[6][:2]))
def test_attention_ignores_what_no_row_sees(case, rot):
    """Slots behind kv_len and in front of the window, whole pages there included (their
    table entries say nothing valid), may hold anything."""
    dt, h, hq, hkv, ps, order, seqs, mode, window = case
    pg = Pages(seqs, hkv, h, ps, dt, order)
    q = rnd(22, pg.n, hq, h, dt=dt)
    flags = flags_of(mode, len(seqs))
    clean = binding.dg_paged_attention(pg.cache, pg.batch, q, causal_arg(mode, flags), window)
    keep = torch.zeros(pg.k.shape[:2], dtype=torch.bool, device="cuda")
    for b, (ql, kv) in enumerate(seqs):
        ranges = [seen_range(ql, kv, flags[b], window, i) for i in range(ql)]
        ranges = [r for r in ranges if r[1] > r[0]]
        lo = min([r[0] for r in ranges], default=0)
        hi = max([r[1] for r in ranges], default=0)
        keep[pg.slots(b, lo, hi)] = True
        for i in range(pg.table.shape[1]):
            if hi <= lo or (i + 1) * ps <= lo or i * ps >= hi:
                pg.table[b, i] = 1 << 30 if i % 2 else -1
    pg.k[~keep], pg.v[~keep] = rot, rot
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = binding.dg_paged_attention(pg.cache, pg.batch, q, causal_arg(mode, flags), window,
                                     err=err)
    binding.dg_paged_check(err)
    assert torch.equal(got, clean)


def test_attention_bad_pages_give_nan_rows_and_bad_lengths_nothing():
    pg = Pages([(1, 300), (40, 200), (2, 500), (1, 64)], 2, 64, 16, BF16)
    q = rnd(23, pg.n, 4, 64)
    clean = binding.dg_paged_attention(pg.cache, pg.batch, q)
    pg.table[0, 3] = pg.k.shape[0]
    pg.table[2, 30] = -1
    pg.kv_len[3] = -1
    out = torch.full_like(clean, 7.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.dg_paged_attention(pg.cache, pg.batch, q, out=out, err=err)
    assert int(err) == binding.PAGED_BAD_BATCH | binding.PAGED_BAD_PAGE
    assert torch.equal(out[1:41], clean[1:41]) and bool((out[43:] == 7).all())
    assert bool(out[0].isnan().all()) and bool(out[41:43].isnan().all())
    # chunk bounds outside the rows, decreasing, or longer than max_q: those sequences' rows
    # are left as they were
    for bad, left in (([0, 1, 41, 43, 45], slice(43, 44)), ([-3, 1, 41, 43, 44], slice(0, 1)),
                      ([0, 43, 41, 43, 44], slice(0, 1))):
        fresh = Pages(pg.seqs, 2, 64, 16, BF16)
        fresh.q_start.copy_(torch.tensor(bad, dtype=torch.int32))
        out.fill_(7.0)
        err.zero_()
        binding.dg_paged_attention(fresh.cache, fresh.batch, q, out=out, err=err)
        assert int(err) == binding.PAGED_BAD_BATCH
        assert bool((out[left] == 7).all())


def test_graph_replays_follow_the_device_tensors_and_streams_do_not_mix():
    """append + attention captured once; lengths, tables and rows change between replays.
    Two such graphs replay at once on two streams."""
    dt, hq, hkv, h, ps = BF16, 8, 2, 64, 16
    rope = binding.dg_rope_init(1e4, h)
    sets = []
    for seed in (1, 2):
        pg = Pages([(1, 60), (1, 61), (1, 62)], hkv, h, ps, dt, seed=seed)
        x = rnd(seed, 3, hq + 2 * hkv, h)
        sets.append((pg, x, torch.empty(3, hq, h, dtype=dt, device="cuda"),
                     torch.empty(3, hq, h, dtype=dt, device="cuda")))

    def step(pg, x, qo, out, stream=None):
        binding.dg_paged_append(pg.cache, pg.batch, x[:, hq:hq + hkv], x[:, hq + hkv:], rope,
                                None, 1e-6, x[:, :hq], None, qo, stream=stream)
        binding.dg_paged_attention(pg.cache, pg.batch, qo, window=50, out=out, stream=stream)

    for s in sets:
        step(*s)
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*s)
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for round_ in range(4):
        for pg, x, qo, out in sets:
            x.copy_(rnd(50 + round_, *x.shape))
            pg.kv_len.sub_(7)
        want = []
        for pg, x, qo, out in sets:
            keep = pg.kmem.clone(), pg.vmem.clone()
            step(pg, x, qo, out)
            want.append(out.clone())
            pg.kmem.copy_(keep[0]), pg.vmem.copy_(keep[1])
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
        torch.cuda.synchronize()
        for (pg, x, qo, out), w in zip(sets, want):
            assert torch.equal(out, w)
    # eager calls on a stream of the caller's
    pg, x, qo, out = sets[0]
    out.zero_()
    torch.cuda.synchronize()
    step(pg, x, qo, out, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(out, want[0])


def test_chunks_append_and_attend_as_one_prompt():
    """The operators in turn, as a serving loop runs them: a prompt in uneven chunks, then
    single tokens, gives the rows of one causal pass; a canvas then sees all of it."""
    dt, hq, hkv, h, ps, total = BF16, 8, 2, 128, 32, 421
    rope = binding.dg_rope_init(1e4, h)
    x = rnd(31, total, hq + 2 * hkv, h)
    one = Pages([(total, total)], hkv, h, ps, dt)
    q1 = binding.dg_paged_append(one.cache, one.batch, x[:, hq:hq + hkv], x[:, hq + hkv:], rope,
                                 None, 1e-6, x[:, :hq])
    qk, kk = binding.dg_qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv],
                                     torch.arange(total, device="cuda", dtype=torch.int32), rope)
    assert torch.equal(q1, qk) and torch.equal(one.k[one.slots(0, 0, total)], kk)
    whole = binding.dg_paged_attention(one.cache, one.batch, q1)
    want, bound, _, _ = attention_fp64(one, q1, [True], 0, h ** -0.5)
    check(whole, want, bound, dt)
    two = Pages([(total, total)], hkv, h, ps, dt, seed=5)
    at = 0
    for c in [200, 129, 1, 64, 7] + [1] * 20:
        start = torch.tensor([0, c], dtype=torch.int32, device="cuda")
        batch = binding.PagedBatch(start, start[1:] + at, two.table, c)
        rows = x[at:at + c]
        q = binding.dg_paged_append(two.cache, batch, rows[:, hq:hq + hkv], rows[:, hq + hkv:],
                                    rope, None, 1e-6, rows[:, :hq])
        part = binding.dg_paged_attention(two.cache, batch, q)
        check(part, want[at:at + c], bound[at:at + c], dt)
        at += c
    assert at == total
    assert torch.equal(two.k[two.slots(0, 0, total)], one.k[one.slots(0, 0, total)])


def test_cache_of_a_model_moves_into_pages():
    """A dg_kv handle's keys (already rotated) and values, copied into pages without norm or
    rotation: a canvas attends to them as the model's own layer does, one softmax over the
    window and the canvas."""
    from gpu_helpers import make_model
    from synth import model_inputs, workloads
    w = workloads.SMALL_BF16
    model = make_model(w)
    kv = binding.dg_prefill(model, model_inputs.prompt(w, "cuda"))
    k, v = binding.dg_kv_read(kv)   # [L, B, Hkv, W, h]
    binding.dg_sync_status(model)
    W, Cn, Bn = kv.W, w.canvas, w.batch
    hkv, hq, h = w.n_kv_heads, w.n_q_heads, w.head_dim
    pg = Pages([(W + Cn, W + Cn)] * Bn, hkv, h, 16, BF16)
    xc = rnd(41, Bn, Cn, hq + 2 * hkv, h)
    rows_k = torch.cat((k[1].transpose(1, 2), xc[:, :, hq:hq + hkv]), 1).reshape(-1, hkv, h)
    rows_v = torch.cat((v[1].transpose(1, 2), xc[:, :, hq + hkv:]), 1).reshape(-1, hkv, h)
    binding.dg_paged_append(pg.cache, pg.batch, rows_k, rows_v)
    canvas = binding.PagedBatch(torch.arange(0, Bn * Cn + 1, Cn, dtype=torch.int32, device="cuda"),
                                pg.kv_len, pg.table, Cn)
    q = xc[:, :, :hq].reshape(-1, hq, h)
    got = binding.dg_paged_attention(pg.cache, canvas, q, causal=False, window=w.window)
    for b in range(Bn):
        kk = rows_k.view(Bn, -1, hkv, h)[b].double().cpu().numpy().transpose(1, 0, 2)
        vv = rows_v.view(Bn, -1, hkv, h)[b].double().cpu().numpy().transpose(1, 0, 2)
        qq = xc[b, :, :hq].double().cpu().numpy()
        for j in range(hq):
            s = qq[:, j] @ kk[j // (hq // hkv)].T / math.sqrt(h)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o = p @ vv[j // (hq // hkv)]
            tol = 2.0 ** -8 * (p @ np.abs(vv[j // (hq // hkv)]) + np.abs(o)) * 1.05
            assert (np.abs(got.view(Bn, Cn, hq, h)[b, :, j].double().cpu().numpy() - o)
                    <= tol).all()
    kv.close()
    model.close()


def test_shared_prefix_pages_and_interleaved_storage():
    """Two sequences whose tables share their first pages read them as one does; keys and
    values may be halves of one tensor; q_out may be q's own rows."""
    dt, hq, hkv, h, ps = BF16, 8, 2, 64, 16
    store = rnd(71, 40, 2, ps, hkv, h)
    cache = binding.PagedCache(store[:, 0], store[:, 1])
    table = torch.tensor([[3, 9, 11, 30, -1], [3, 9, 20, 21, 22]], dtype=torch.int32, device="cuda")
    kv = torch.tensor([50, 70], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1, 3], dtype=torch.int32, device="cuda")
    batch = binding.PagedBatch(start, kv, table, 2)
    x = rnd(72, 3, hq + 2 * hkv, h)
    rope = binding.dg_rope_init(1e4, h)
    apart = x.clone()
    want_q = binding.dg_paged_append(cache, batch, apart[:, hq:hq + hkv], apart[:, hq + hkv:],
                                     rope, None, 1e-6, apart[:, :hq])
    got_q = binding.dg_paged_append(cache, batch, x[:, hq:hq + hkv], x[:, hq + hkv:], rope, None,
                                    1e-6, x[:, :hq], None, x[:, :hq])
    assert got_q.data_ptr() == x.data_ptr() and torch.equal(got_q, want_q)
    both = binding.dg_paged_attention(cache, batch, got_q)
    for b in range(2):
        one = binding.PagedBatch(start[b:b + 2] - start[b], kv[b:b + 1], table[b:b + 1], 2)
        rows = slice(int(start[b]), int(start[b + 1]))
        alone = binding.dg_paged_attention(cache, one, got_q[rows])
        # the split differs with the batch, so the same keys add up in another order: each
        # result is within half a step of sum p|v| for the weights and of itself, both at
        # most the largest |v| (and fp32's share far below the slack of these two bounds)
        tol = 4 * half_step(dt) * float(cache.v_pages.abs().max())
        assert float((alone.double() - both[rows].double()).abs().max()) <= tol


def test_first_call_of_a_process_may_be_captured():
    """Nothing that a capture forbids happens in the first calls (tables of entry points,
    kernel attributes)."""
    import os
    import subprocess
    import sys
    here = os.path.dirname(os.path.abspath(__file__))
    code = """
import sys; sys.path[:0] = [%r, %r]
import torch
from masked_discrete_diffusion_b200 import binding
import test_gpu_paged as t
pg = t.Pages([(1, 60), (3, 61)], 2, 64, 16, torch.bfloat16)
x = t.rnd(1, 4, 8, 64)
rope = binding.dg_rope_init(1e4, 64)
qo = torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda")
out = torch.zeros_like(qo)
def step():
    binding.dg_paged_append(pg.cache, pg.batch, x[:, 4:6], x[:, 6:], rope, None, 1e-6, x[:, :4],
                            None, qo)
    binding.dg_paged_attention(pg.cache, pg.batch, qo, out=out)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
a = out.clone()
out.zero_()
step()
assert torch.equal(a, out) and bool((a != 0).any())
""" % (os.path.dirname(here), here)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("q,length,causal", [(9, 20000, True), (1, 30000, True), (150, 4000, False)])
def test_calls_in_a_row_over_scattered_pages_agree(q, length, causal):
    """The copies of one call land in many orders when its pages lie far apart in memory that no
    cache holds: every call's bits are the first one's, and no wait gives up."""
    hkv, h, ps, b = 4, 128, 32, 16
    pg = Pages([(q, length - 517 * i % 1900) for i in range(b)], hkv, h, ps, BF16, seed=81,
               extra=5000)
    x = rnd(83, pg.n, 8 * hkv, h)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    first = binding.dg_paged_attention(pg.cache, pg.batch, x, causal, err=err)
    assert torch.isfinite(first).all()
    out, flush = torch.empty_like(first), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(200):
        if i % 2:
            flush.fill_(i)
        binding.dg_paged_attention(pg.cache, pg.batch, x, causal, out=out, err=err)
        wrong += (out.view(torch.int16) != first.view(torch.int16)).sum()
    assert int(wrong) == 0
    binding.dg_paged_check(err)
