"""The paged-cache operators, case by case: inputs, plain forms and the framework's calls.

Three operators that a serving loop with a paged key/value cache runs in every layer:

* ``qk_norm_rope``: RMSNorm of every query and key head (gain per channel) and the
  rotation to the row's position, in one pass over the QKV projection's rows;
* ``paged_append``: the chunk's keys (normalised and rotated on the way) and values go
  into the pages of their sequences, the queries to a dense output;
* ``paged_attention``: each sequence's chunk of new tokens attends to its pages, causally
  or in both directions inside the chunk, with or without a sliding window.

``run`` computes them in elementary torch operations in 32 bits (angles in 64), or, with
``own`` set, through ``masked_discrete_diffusion_b200.binding``.  ``exact`` is a separate
64-bit form.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
BASE = 10000.0


# ---------------------------------------------------------------------------- cases
def _norm(name, n, hq, hkv, h, dtype, far):
    """n rows of hq + hkv heads; positions are drawn below `far`."""
    return {"name": name, "op": "qk_norm_rope", "n": n, "hq": hq, "hkv": hkv, "h": h,
            "dtype": dtype, "far": far}


def _paged(name, op, b, q, ctx, hq, hkv, h, dtype, page, lens, mode="causal", window=0, pad=0):
    """b sequences with chunks of up to q new tokens after up to ctx cached ones.

    lens 0: every sequence has exactly q and ctx; else both are drawn (over their
    logarithm) from that seed, the first sequence keeping the full sizes.  mode: "causal",
    "both" (bidirectional inside the chunk) or "mixed" (a flag per sequence, every chunk a
    whole block of q rows).  pad: rows
    behind the last sequence, which the calls leave alone."""
    return {"name": name, "op": op, "b": b, "q": q, "ctx": ctx, "hq": hq, "hkv": hkv, "h": h,
            "dtype": dtype, "page": page, "lens": lens, "mode": mode, "window": window,
            "pad": pad}


def listed():
    return [
        # one token of one sequence: the launch is all there is
        _norm("norm-one-token", 1, 16, 8, 128, "bf16", 1024),
        # a forward over eight canvases of 256 rows after 8,192-token prompts
        _norm("norm-canvases", 2048, 16, 8, 128, "bf16", 8448),
        # a long prompt of a small-head model in half precision, at far positions
        _norm("norm-long-f16", 32767, 32, 4, 64, "f16", 1 << 20),
        # single-token serving: every sequence of a batch adds one key and one value
        _paged("append-tokens", "paged_append", 64, 1, 8191, 16, 8, 128, "bf16", 16, 0),
        # prompts of mixed lengths packed into one pass, with padding rows behind them
        _paged("append-prompts", "paged_append", 16, 4096, 2048, 16, 8, 128, "bf16", 64, 11,
               pad=61),
        # single-token serving of one short sequence: the smallest call
        _paged("attend-one-token", "paged_attention", 1, 1, 1023, 16, 8, 128, "bf16", 64, 0),
        # single-token serving of a full batch with long caches of unequal lengths
        _paged("attend-tokens", "paged_attention", 64, 1, 16383, 32, 8, 128, "bf16", 16, 5),
        # eight canvases denoised against the last 1,024 positions of long prompts
        _paged("attend-canvases", "paged_attention", 8, 256, 8192, 16, 8, 128, "bf16", 64, 0,
               mode="both", window=1024),
        # one long prompt in one chunk, every earlier position visible
        _paged("attend-prompt", "paged_attention", 1, 8192, 0, 16, 8, 128, "bf16", 128, 0),
        # a small-head model's prompts in half precision, odd lengths, sliding window
        _paged("attend-windowed-f16", "paged_attention", 7, 2047, 1500, 12, 4, 64, "f16", 32, 3,
               window=1000, pad=5),
        # some sequences append finished blocks (causal) while others denoise (both ways)
        _paged("attend-mixed", "paged_attention", 24, 256, 4096, 16, 8, 128, "bf16", 64, 9,
               mode="mixed"),
        # drafted tokens being checked: short chunks after long caches, many heads a key
        _paged("attend-drafts", "paged_attention", 16, 9, 20000, 32, 4, 128, "bf16", 32, 8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "paged_append", "paged_attention", "paged_attention"])
    h = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 7, 8])
    if op == "qk_norm_rope":
        dtype = rng.choice(["bf16", "f16", "f32"])
        n = _log(rng, 1, 32767 * 36 * 64 // ((hq + hkv) * h * (2 if dtype == "f32" else 1)))
        c = _norm("", min(n, 40000), hq, hkv, h, dtype, _log(rng, 64, 1 << 20))
    else:
        dtype = rng.choice(["bf16", "f16"])
        page = rng.choice([16, 32, 64, 128, 256])
        b, q, ctx = _log(rng, 1, 64), _log(rng, 1, 4096), _log(rng, 1, 16384)
        mode = rng.choice(["causal", "both", "mixed"])
        window = rng.choice([0, 0, 128, 1000, 1024])
        c = _paged("", op, b, q, ctx, hq, hkv, h, dtype, page, rng.randrange(1, 1 << 30), mode,
                   window, rng.choice([0, 0, 3, 64]))
        # no dearer than the largest listed case of its kind, in rows and in score entries
        while c["b"] * c["q"] > 16384 or c["b"] * (c["q"] + c["ctx"]) * c["hkv"] * h > 2 ** 30 or (
                op == "paged_attention"
                and c["b"] * c["q"] * (c["q"] + c["ctx"]) * c["hq"] > 2 ** 29):
            big = max(("b", "q", "ctx"), key=lambda k: c[k] if k != "b" else c[k] * 16)
            c[big] = max(1, c[big] * 3 // 4)
    del c["name"]
    return c


def _lens(case):
    """Chunk length and cached length of every sequence (from the case alone)."""
    b, q, ctx = case["b"], case["q"], case["ctx"]
    if not case["lens"]:
        return [q] * b, [ctx] * b
    rng = random.Random(case["lens"])
    low = q if case["mode"] == "mixed" else max(1, q // 16)  # mixed: whole blocks
    qs = [q] + [_log(rng, low, q) for _ in range(b - 1)]
    cs = [ctx] + [_log(rng, max(1, ctx // 64), ctx) if ctx else 0 for _ in range(b - 1)]
    return qs, cs


def _flags(case):
    """Whether each sequence is causal."""
    if case["mode"] == "mixed":
        return [(i % 3) != 1 for i in range(case["b"])]
    return [case["mode"] == "causal"] * case["b"]


# ---------------------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, hq, hkv, h = DTYPES[case["dtype"]], case["hq"], case["hkv"], case["h"]
    s = {"case": dict(case)}

    def rows(n):  # a QKV projection's output and its three views
        x = torch.randn(n, hq + 2 * hkv, h, generator=gen, device=dev).to(dt)
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]

    if case["op"] != "paged_attention":
        s["q_gain"] = (1 + 0.1 * torch.randn(h, generator=gen, device=dev)).to(dt)
        s["k_gain"] = (1 + 0.1 * torch.randn(h, generator=gen, device=dev)).to(dt)
    if case["op"] == "qk_norm_rope":
        n = case["n"]
        s["q"], s["k"], _ = rows(n)
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=dev,
                                       dtype=torch.int32)
        if own:
            from masked_discrete_diffusion_b200 import binding
            s["rope"] = binding.dg_rope_init(BASE, h)
        return s
    qs, cs = _lens(case)
    ps, b = case["page"], case["b"]
    n = sum(qs) + case["pad"]
    need = [-(-(c + q) // ps) for q, c in zip(qs, cs)]
    pages = sum(need) + 3
    s["k_pages"] = torch.randn(pages, ps, hkv, h, generator=gen, device=dev).to(dt)
    s["v_pages"] = torch.randn(pages, ps, hkv, h, generator=gen, device=dev).to(dt)
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    width = max(need)
    at = torch.arange(width, device=dev)[None, :]
    first = torch.tensor([sum(need[:i]) for i in range(b)], device=dev)[:, None]
    used = at < torch.tensor(need, device=dev)[:, None]
    table = torch.where(used, perm[(first + at).clamp(max=pages - 1)], torch.full_like(perm[:1], -1))
    s["page_table"] = table.to(torch.int32).contiguous()
    start = [0]
    for q in qs:
        start.append(start[-1] + q)
    s["q_start"] = torch.tensor(start, dtype=torch.int32, device=dev)
    s["kv_len"] = torch.tensor([q + c for q, c in zip(qs, cs)], dtype=torch.int32, device=dev)
    s["max_q"] = max(qs)
    q, k, v = rows(n)
    s["q"] = q
    s["out"] = torch.zeros(n, hq, h, dtype=dt, device=dev)
    if case["op"] == "paged_append":
        s["k"], s["v"] = k, v
    else:
        s["causal"] = torch.tensor(_flags(case), dtype=torch.uint8, device=dev)
    if own:
        from masked_discrete_diffusion_b200 import binding
        s["rope"] = binding.dg_rope_init(BASE, h)
        s["cache"] = binding.PagedCache(s["k_pages"], s["v_pages"])
        s["batch"] = binding.PagedBatch(s["q_start"], s["kv_len"], s["page_table"], s["max_q"])
    return s


# ---------------------------------------------------------------------------- plain forms
def _turn(x, gain, positions):
    """RMSNorm of the last axis times gain, then the rotation of pairs (i, i + h/2) by
    position * base^(-2i/h); in 32 bits, the angles in 64.  x [n, heads, h]."""
    h = x.shape[-1]
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gain.float()
    inv = BASE ** (-torch.arange(0, h, 2, device=x.device, dtype=torch.float64) / h)
    a = positions.double()[:, None] * inv
    c, s = a.cos().float()[:, None, :], a.sin().float()[:, None, :]
    u, w = y[..., :h // 2], y[..., h // 2:]
    return torch.cat((u * c - w * s, w * c + u * s), -1).to(x.dtype)


def _rows(s):
    """Per row of the chunks: its sequence and its position."""
    q_start, n = s["q_start"].long(), int(s["q"].shape[0]) - s["case"]["pad"]
    i = torch.arange(n, device=q_start.device)
    b = torch.searchsorted(q_start[1:], i, right=True)
    past = s["kv_len"].long() - (q_start[1:] - q_start[:-1])
    return b, past[b] + i - q_start[b]


def _plain_append(s):
    b, pos = _rows(s)
    n, ps = pos.shape[0], s["case"]["page"]
    page = s["page_table"].long()[b, pos // ps]
    s["k_pages"][page, pos % ps] = _turn(s["k"][:n], s["k_gain"], pos)
    s["v_pages"][page, pos % ps] = s["v"][:n]
    s["out"][:n] = _turn(s["q"][:n], s["q_gain"], pos)
    return {"k": s["k_pages"], "v": s["v_pages"], "q": s["out"]}


def _plain_attention(s):
    c = s["case"]
    hq, hkv, h, ps, window = c["hq"], c["hkv"], c["h"], c["page"], c["window"]
    q_start, kv_len = s["q_start"].long(), s["kv_len"].long()
    dev, nb, mq = q_start.device, c["b"], s["max_q"]
    q_len = q_start[1:] - q_start[:-1]
    i = torch.arange(mq, device=dev)
    row = q_start[:-1, None] + torch.minimum(i[None], (q_len - 1)[:, None])      # [b, mq]
    q = s["q"][row].float().reshape(nb, mq, hkv, hq // hkv, h).permute(0, 2, 3, 1, 4)
    width = s["page_table"].shape[1] * ps
    j = torch.arange(width, device=dev)
    page = s["page_table"].long().clamp(min=0)[:, j // ps]                       # [b, width]
    k = s["k_pages"][page, j % ps].float().permute(0, 2, 1, 3)                   # [b, hkv, width, h]
    v = s["v_pages"][page, j % ps].float().permute(0, 2, 1, 3)
    past = (kv_len - q_len)[:, None, None]
    pos = past + i[None, :, None]
    causal = s["causal"].bool()[:, None, None]
    seen = (j < kv_len[:, None, None]) & ((j <= pos) | ~causal)
    if window:
        seen &= j >= torch.where(causal, pos - window + 1, past - window)
    g = hq // hkv
    p = (q.reshape(nb, hkv, g * mq, h) @ k.transpose(-1, -2)).mul_(1 / math.sqrt(h))
    p = p.view(nb, hkv, g, mq, width).masked_fill_(~seen[:, None, None], -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True)).view(nb, hkv, g * mq, width)
    o = (p @ v).view(nb, hkv, g, mq, h).permute(0, 3, 1, 2, 4).reshape(nb, mq, hq, h)
    s["out"][row[i[None] < q_len[:, None]]] = o[i[None] < q_len[:, None]].to(s["out"].dtype)
    return s["out"]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        if op == "qk_norm_rope":
            return (_turn(s["q"], s["q_gain"], s["positions"]),
                    _turn(s["k"], s["k_gain"], s["positions"]))
        return _plain_append(s) if op == "paged_append" else _plain_attention(s)
    from masked_discrete_diffusion_b200 import binding
    if op == "qk_norm_rope":
        return binding.dg_qk_norm_rope(s["q"], s["k"], s["positions"], s["rope"],
                                       q_gain=s["q_gain"], k_gain=s["k_gain"], eps=EPS)
    if op == "paged_append":
        binding.dg_paged_append(s["cache"], s["batch"], s["k"], s["v"], s["rope"],
                                k_gain=s["k_gain"], eps=EPS, q=s["q"], q_gain=s["q_gain"],
                                q_out=s["out"])
        return {"k": s["k_pages"], "v": s["v_pages"], "q": s["out"]}
    return binding.dg_paged_attention(s["cache"], s["batch"], s["q"], causal=s["causal"],
                                      window=s["case"]["window"], out=s["out"])


# ---------------------------------------------------------------------------- 64 bits
def _exact_head(x, gain, pos):
    """x [n, h] float64, pos [n] float64: norm, gain, rotation as a complex product."""
    h = x.shape[-1]
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / h + EPS) * gain
    e = torch.exp(-math.log(BASE) * 2 / h * torch.arange(h // 2, device=x.device,
                                                         dtype=torch.float64))
    z = torch.complex(x[:, :h // 2], x[:, h // 2:])
    a = pos[:, None] * e[None]
    z = z * torch.polar(torch.ones_like(a), a)
    return torch.cat((z.real, z.imag), 1)


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, h = case["hq"], case["hkv"], case["h"]
    if case["op"] == "qk_norm_rope":
        pos = s["positions"].double()
        return tuple(torch.stack([_exact_head(x[:, j].double(), gain.double(), pos)
                                  for j in range(x.shape[1])], 1)
                     for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])))
    start, total, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["page_table"].long()
    ps = case["page"]
    if case["op"] == "paged_append":
        kp, vp, out = s["k_pages"].double(), s["v_pages"].double(), s["out"].double()
        for b in range(case["b"]):
            lo, hi = start[b], start[b + 1]
            pos = torch.arange(total[b] - (hi - lo), total[b], device="cuda")
            at = table[b, pos // ps] * ps + pos % ps
            p64 = pos.double()
            for j in range(hkv):
                kp.view(-1, hkv, h)[at, j] = _exact_head(s["k"][lo:hi, j].double(),
                                                         s["k_gain"].double(), p64)
            vp.view(-1, hkv, h)[at] = s["v"][lo:hi].double()
            for j in range(hq):
                out[lo:hi, j] = _exact_head(s["q"][lo:hi, j].double(), s["q_gain"].double(), p64)
        return {"k": kp, "v": vp, "q": out}
    out, flags, w = s["out"].double(), _flags(case), case["window"]
    for b in range(case["b"]):
        lo, hi = start[b], start[b + 1]
        past = total[b] - (hi - lo)
        first = max(0, past - w) if w else 0  # nothing of the chunk sees further back
        j = torch.arange(first, total[b], device="cuda")
        at = table[b, j // ps] * ps + j % ps
        for g in range(hkv):
            k = s["k_pages"].view(-1, hkv, h)[at, g].double()
            v = s["v_pages"].view(-1, hkv, h)[at, g].double()
            for c0 in range(lo, hi, 1024):
                c1 = min(hi, c0 + 1024)
                i = past + torch.arange(c0 - lo, c1 - lo, device="cuda")[:, None]
                hide = torch.zeros(c1 - c0, j.shape[0], dtype=torch.bool, device="cuda")
                if flags[b]:
                    hide |= j[None] > i
                    if w:
                        hide |= i - j[None] >= w
                elif w:
                    hide |= (j < past - w)[None]
                for r in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                    x = s["q"][c0:c1, r].double() @ k.T / math.sqrt(h)
                    out[c0:c1, r] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ v
    return out


# ---------------------------------------------------------------------------- work
def work(case):
    hq, hkv, h = case["hq"], case["hkv"], case["h"]
    size = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    if case["op"] == "qk_norm_rope":
        # rows read and written once, positions and gains read; per element a square, a
        # scaling, the gain and the rotation's products
        n = case["n"]
        return {"bytes": 2 * n * (hq + hkv) * h * size + 4 * n + 2 * h * size,
                "flops": 9 * n * (hq + hkv) * h}
    qs, cs = _lens(case)
    n = sum(qs)
    ps = case["page"]
    if case["op"] == "paged_append":
        pages = sum((q + c - 1) // ps - c // ps + 1 for q, c in zip(qs, cs))
        return {"bytes": 2 * n * (hq + 2 * hkv) * h * size + 4 * (pages + 2 * case["b"]),
                "flops": 9 * n * (hq + hkv) * h}
    pairs = keys = 0
    w = case["window"]
    for q, c, causal in zip(qs, cs, _flags(case)):
        back = min(c, w) if w else c
        if not causal:
            pairs += q * (back + q)
            keys += back + q
        elif not w:
            pairs += q * c + q * (q + 1) // 2
            keys += c + q
        else:
            pairs += sum(min(c + i + 1, w) for i in range(q))
            keys += min(c, w - 1) + q
    return {"bytes": (2 * n * hq + 2 * keys * hkv) * h * size + 4 * keys // ps,
            "flops": 4 * pairs * hq * h}
