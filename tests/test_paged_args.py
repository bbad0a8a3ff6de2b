"""Refusals of the paged-cache operators, which come before any CUDA call (no GPU): the C
entry points on fake pointers, the binding on host tensors, and the rotation's constants."""
import ctypes
import math
import os
import re
from fractions import Fraction

import pytest
import torch

from masked_discrete_diffusion_b200 import binding, build

BF16, F16, F32 = 0, 1, 2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 4096  # never dereferenced: every call below is refused


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, dtype=BF16, n_pages=4, page_size=16, n_kv_heads=2, head_dim=64,
             page_stride=16 * 2 * 64, token_stride=2 * 64, head_stride=64)
    a.update(kw)
    return binding.dg_paged_cache(**a)


def batch(**kw):
    a = dict(B=2, n_tokens=3, max_q=2, max_pages=4, q_start=FAKE, kv_len=FAKE, page_table=FAKE)
    a.update(kw)
    return binding.dg_paged_batch(**a)


def heads(n=2, **kw):
    a = dict(p=FAKE, token_stride=64 * n, head_stride=64, n_heads=n)
    a.update(kw)
    return binding.dg_heads(**a)


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope(h=64):
    return binding.dg_rope_init(10000.0, h)


def attention(lib, c=None, b=None, q=None, causal=1, window=0, scale=0.125, out=FAKE, lse=None,
              ws=FAKE, ws_bytes=1 << 40, err=None):
    return lib.dg_paged_attention(ref(c or cache()), ref(b or batch()), ref(q or heads(4)), causal,
                                  None, window, scale, out, lse, ws, ws_bytes, err, None)


def append(lib, c=None, b=None, k=None, v=None, r=None, kg=None, eps=-1.0, q=None, qg=None,
           qo=None, err=None):
    return lib.dg_paged_append(ref(c or cache()), ref(b or batch()), ref(k or heads()),
                               ref(v or heads()), ref(r), kg, eps, ref(q), qg, ref(qo), err, None)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=FAKE + 8), dict(dtype=F32), dict(dtype=7),
              dict(n_pages=0), dict(page_size=8), dict(page_size=24), dict(page_size=1 << 21),
              dict(n_kv_heads=0), dict(head_dim=0), dict(head_dim=72), dict(head_dim=272),
              dict(page_stride=0), dict(token_stride=0), dict(head_stride=32),
              dict(head_stride=68), dict(token_stride=64), dict(page_stride=1 << 39),
              dict(page_stride=16 * 2 * 64 - 8)]
BAD_BATCHES = [dict(B=-1), dict(n_tokens=-1), dict(max_q=-1), dict(max_pages=-1),
               dict(max_pages=1 << 28), dict(q_start=None), dict(kv_len=None),
               dict(page_table=None), dict(kv_len=FAKE + 2)]
BAD_HEADS = [dict(p=None), dict(p=FAKE + 8), dict(token_stride=-64), dict(token_stride=68),
             dict(head_stride=60), dict(head_stride=1 << 41), dict(n_heads=-1)]


@pytest.mark.parametrize("bad", BAD_CACHES, ids=str)
def test_caches_refused(lib, bad):
    assert attention(lib, c=cache(**bad)) == 1 and lib.dg_last_error()
    assert append(lib, c=cache(**bad)) == 1 and lib.dg_last_error()
    n = ctypes.c_size_t()
    assert lib.dg_paged_attention_workspace(ref(cache(**bad)), ref(batch()), 4, ctypes.byref(n)) == 1


@pytest.mark.parametrize("bad", BAD_BATCHES, ids=str)
def test_batches_refused(lib, bad):
    assert attention(lib, b=batch(**bad)) == 1 and lib.dg_last_error()
    assert append(lib, b=batch(**bad)) == 1 and lib.dg_last_error()


@pytest.mark.parametrize("bad", BAD_HEADS, ids=str)
def test_heads_refused(lib, bad):
    assert attention(lib, q=heads(4, **bad)) == 1 and lib.dg_last_error()
    assert append(lib, k=heads(**bad)) == 1 and append(lib, v=heads(**bad)) == 1
    assert append(lib, q=heads(4, **bad), qo=heads(4)) == 1
    assert append(lib, q=heads(4), qo=heads(4, **bad)) == 1


def test_attention_arguments_refused(lib):
    for bad in (dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.inf),
                dict(scale=math.nan), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2),
                dict(err=FAKE + 1), dict(ws=None), dict(ws=FAKE + 16), dict(ws_bytes=16),
                dict(q=heads(3)), dict(q=heads(0))):
        assert attention(lib, **bad) == 1, bad
        assert lib.dg_last_error()
    # shapes that are valid but not built
    wide = cache(head_dim=96, page_stride=16 * 2 * 96, token_stride=2 * 96, head_stride=96)
    assert attention(lib, c=wide) == 2 and b"head_dim" in lib.dg_last_error()
    assert attention(lib, q=heads(2 * 129)) == 2 and b"128" in lib.dg_last_error()
    # one row of q may have any stride; more need their own memory
    for kw in (dict(token_stride=0), dict(head_stride=0)):
        assert attention(lib, q=heads(4, **kw)) == 1 and b"strides of 0" in lib.dg_last_error()
    # a line of key tiles that 32 bits could not count
    huge = batch(B=1 << 20, n_tokens=1 << 30, max_q=1 << 20, max_pages=1 << 22)
    assert attention(lib, b=huge, q=heads(4)) == 2 and b"too many" in lib.dg_last_error()


def test_append_arguments_refused(lib):
    for bad in (dict(k=heads(3)), dict(v=heads(1)), dict(q=heads(4)), dict(qo=heads(4)),
                dict(kg=FAKE), dict(eps=1e-6, kg=FAKE + 8), dict(eps=math.nan),
                dict(eps=math.inf), dict(eps=1e-6, qg=FAKE), dict(r=rope(128)),
                dict(q=heads(4), qo=heads(2)), dict(err=FAKE + 1),
                dict(q=heads(4), qo=heads(4, head_stride=0)),
                dict(q=heads(4), qo=heads(4, token_stride=64))):
        assert append(lib, **bad) == 1, bad
        assert lib.dg_last_error()


def test_norm_rope_arguments_refused(lib):
    def call(dtype=BF16, n=3, h=64, q=None, k=None, pos=FAKE, r=None, qg=None, kg=None, eps=1e-6,
             qo=None, ko=None):
        return lib.dg_qk_norm_rope(dtype, n, h, ref(q or heads(4)), ref(k or heads()), pos,
                                   ref(r or rope()), qg, kg, eps, ref(qo or heads(4)),
                                   ref(ko or heads()), None)

    for bad in (dict(dtype=3), dict(n=-1), dict(h=8), dict(h=72), dict(h=128), dict(pos=None),
                dict(pos=FAKE + 2), dict(qo=heads(2)), dict(eps=math.nan),
                dict(eps=-1.0, qg=FAKE), dict(kg=FAKE + 2), dict(qo=heads(4, head_stride=0)),
                dict(q=heads(4, p=None)), dict(dtype=F32, q=heads(4, head_stride=66))):
        assert call(**bad) == 1, bad
        assert lib.dg_last_error()
    assert lib.dg_qk_norm_rope(BF16, 3, 64, None, ref(heads()), FAKE, None, None, None, 1e-6,
                               ref(heads()), ref(heads()), None) == 1


def test_empty_calls_need_no_device(lib):
    assert attention(lib, b=batch(n_tokens=0)) == 0 and attention(lib, b=batch(B=0)) == 0
    assert append(lib, b=batch(n_tokens=0)) == 0 and append(lib, b=batch(B=0)) == 0
    n = ctypes.c_size_t()
    assert lib.dg_paged_attention_workspace(ref(cache()), ref(batch()), 4, ctypes.byref(n)) == 0
    assert lib.dg_paged_attention_workspace(ref(cache()), ref(batch()), 3, ctypes.byref(n)) == 1
    assert lib.dg_paged_attention_workspace(ref(cache()), ref(batch()), 4, None) == 1


def header_fields(name):
    """(type, field) of a struct of dg_paged.h, in order; pointers as "*"."""
    src = open(os.path.join(ROOT, "include", "dg_paged.h")).read()
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), src, re.S).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    out = []
    for decl in body.split(";"):
        m = re.match(r"\s*(?:const\s+)?(\w+)\s*(.+)", decl.strip(), re.S)
        for f in m.group(2).split(",") if m else ():
            f = f.strip()
            out.append(("*" if f.startswith("*") else m.group(1), re.sub(r"[*\s]|\[.*", "", f)))
    return out


@pytest.mark.parametrize("name", ["dg_heads", "dg_rope", "dg_paged_cache", "dg_paged_batch"])
def test_structs_match_the_header(name):
    """Field order, names and types: one out of place would hand the library a wrong pointer."""
    kinds = {"*": ctypes.c_void_p, "int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64,
             "uint64_t": ctypes.c_uint64 * 128}
    want = [(f, kinds[t]) for t, f in header_fields(name)]
    assert getattr(binding, name)._fields_ == want and len(want) >= 3


def test_rope_constants(lib):
    r = rope(64)
    assert r.head_dim == 64 and all(t == 0 for t in r.turns[32:])
    for i in range(32):
        # fp64 holds the fraction of a turn to 2^-50 of itself (the exponent, the power and
        # the quotient round once each), and the constant is cut to a multiple of 2^-64
        want = 10000.0 ** (-2 * i / 64) / (2 * math.pi)
        assert abs(Fraction(r.turns[i], 1 << 64) - Fraction(want)) <= (
            Fraction(want) / (1 << 50) + Fraction(1, 1 << 64))
    assert binding.dg_rope_init(1.0, 256).turns[127] == binding.dg_rope_init(1.0, 256).turns[0]
    for base, h in ((0.5, 64), (math.nan, 64), (math.inf, 64), (10.0, 8), (10.0, 20), (10.0, 272)):
        with pytest.raises(binding.DGError):
            binding.dg_rope_init(base, h)
    assert lib.dg_rope_init(10000.0, 64, None) == 1


def test_binding_refuses_host_and_misshaped_tensors():
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        binding.dg_qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="3-D"):
        binding.dg_qk_norm_rope(x[0], x)
    with pytest.raises(ValueError, match="3-D"):
        binding.dg_qk_norm_rope(x.double(), x)
    with pytest.raises(ValueError, match="tensor"):
        binding.dg_qk_norm_rope([1], x)
    pages = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="current device"):
        binding.PagedCache(pages, pages)
    with pytest.raises(ValueError, match="4-D"):
        binding.PagedCache(pages.float(), pages.float())
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="current device"):
        binding.PagedBatch(t[0, :3], t[0, :2], t, 1)
    with pytest.raises(ValueError, match="2-D"):
        binding.PagedBatch(t[0, :3], t[0, :2], t.long(), 1)
    with pytest.raises(ValueError, match="eps"):
        binding._eps(float("nan"))
    with pytest.raises(ValueError, match="err"):
        binding.dg_paged_check(torch.zeros(2, dtype=torch.int32))
