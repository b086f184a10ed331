"""Cases and plain forms of the operators of a sparse decode step over the INT4 paged cache.

* ``norm_rope``  norms of q and k per head, rotary positions, then the rotated, quantized append
* ``summary``    the mean key of every page that a step completed, held like a cache row
* ``select``     the pages that a query attends over, by the scores of their mean keys
* ``sparse``     decode attention over each kv-head's own list of pages

``run`` computes the plain form with elementary torch operations, or with ``own`` set makes the
library's calls.  Caches and summaries come back as their bytes: the rules fix every scale, zero
and code to the bit, so they are whole numbers that have to be equal, and so are the lists of pages.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ----------------------------------------------------------------- cases

def listed():
    return [
        # one decoding request: latency
        dict(name="norm-rope-1", op="norm_rope", tokens=1, hq=32, hkv=8, d=128, page=16, rope_dim=128, inter=False,
             h=128, rot_v=False, dt="bf16", meta="f16", wdt="in", offset=0.0, max_pos=32768, chunk=False),
        # a decode step of 256 requests, padded rows among them, weights kept in 32 bits as 1 + w
        dict(name="norm-rope-256", op="norm_rope", tokens=256, hq=64, hkv=8, d=128, page=16, rope_dim=128, inter=True,
             h=128, rot_v=True, dt="bf16", meta="f16", wdt="f32", offset=1.0, max_pos=32768, chunk=False),
        # the long prompt: 131072 tokens at once
        dict(name="norm-rope-131072", op="norm_rope", tokens=131072, hq=32, hkv=8, d=128, page=64, rope_dim=128,
             inter=False, h=128, rot_v=True, dt="bf16", meta="f16", wdt="in", offset=0.0, max_pos=131072, chunk=True),
        # a decode step of 256 requests: about one in 16 completes a page
        dict(name="summary-256", op="summary", seqs=256, lo=2048, hi=4096, new=1, hkv=8, d=128, page=16, meta="f16"),
        # odd chunks of 37 prompts, head_dim 256, 64-token pages
        dict(name="summary-37-chunks", op="summary", seqs=37, lo=1, hi=6000, new=2047, hkv=4, d=256, page=64,
             meta="bf16"),
        # a whole prompt of 131072 tokens
        dict(name="summary-131072", op="summary", seqs=1, lo=131072, hi=131072, new=131072, hkv=8, d=128, page=16,
             meta="f16"),
        # one request with 32768 tokens, 128 pages of them: latency
        dict(name="select-1x32768", op="select", seqs=1, lo=32768, hi=32768, hq=32, hkv=8, d=128, page=16, h=128,
             take=128, first=1, last=4, dt="bf16", meta="f16"),
        # 64 requests up to 16384 tokens, some of them short enough to be taken whole
        dict(name="select-64x16384", op="select", seqs=64, lo=500, hi=16384, hq=32, hkv=8, d=128, page=16, h=128,
             take=128, first=1, last=8, dt="bf16", meta="f16"),
        # 16 requests with 131072 tokens each, 64 q-heads
        dict(name="select-16x131072", op="select", seqs=16, lo=131000, hi=131072, hq=64, hkv=8, d=128, page=16, h=128,
             take=256, first=4, last=16, dt="bf16", meta="f16"),
        # one request, 128 of its pages: latency
        dict(name="sparse-1x2048", op="sparse", seqs=1, lo=32768, hi=32768, take=128, hq=32, hkv=8, d=128, page=16,
             h=128, rot_v=True, dt="bf16", meta="f16"),
        # 37 requests of odd lengths, head_dim 64, 64-token pages
        dict(name="sparse-37x4096", op="sparse", seqs=37, lo=100, hi=20000, take=64, hq=12, hkv=2, d=64, page=64,
             h=64, rot_v=True, dt="f16", meta="bf16"),
        # 256 requests up to 8192 tokens, 128 pages of each, 64 q-heads
        dict(name="sparse-256x2048", op="sparse", seqs=256, lo=2048, hi=8192, take=128, hq=64, hkv=8, d=128, page=16,
             h=128, rot_v=True, dt="bf16", meta="f16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "summary", "select", "sparse"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 64])
    dt, meta = rng.choice(["bf16", "f16"]), rng.choice(["f16", "f16", "bf16"])
    h = rng.choice([x for x in (16, 32, 64, 128, 256) if x <= d])
    if op == "norm_rope":
        tokens = _log_int(rng, 1, max(2, min(60000, 60000 * 1024 // (hkv * d))))
        return dict(op=op, tokens=tokens, hq=hkv * rng.randint(1, 8 if tokens < 20000 else 4), hkv=hkv, d=d, page=page,
                    rope_dim=16 * rng.randint(1, d // 16) if rng.random() < 0.5 else d, inter=rng.random() < 0.5, h=h,
                    rot_v=rng.random() < 0.6, dt=dt, meta=meta, wdt=rng.choice(["in", "f32"]),
                    offset=rng.choice([0.0, 1.0]), max_pos=rng.choice([32768, 131072]), chunk=tokens > 512)
    if op == "summary":
        seqs = _log_int(rng, 1, 512)
        hi = _log_int(rng, 16, 131072 * 1024 // (hkv * d * seqs) if hkv * d > 1024 else max(16, 131072 // seqs))
        return dict(op=op, seqs=seqs, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi,
                    new=rng.choice([1, 1, 5, page, hi, hi]), hkv=hkv, d=d, page=page, meta=meta)
    if op == "select":
        seqs = _log_int(rng, 1, 128)
        hi = _log_int(rng, 64, min(262144, 2000000 * page // 16 // seqs))
        first, last = rng.choice([0, 1, 4]), rng.choice([1, 2, 16])
        return dict(op=op, seqs=seqs, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi, hq=hkv * rng.randint(1, 8),
                    hkv=hkv, d=d, page=page, h=h, take=first + last + _log_int(rng, 1, 512), first=first, last=last,
                    dt=dt, meta=meta)
    seqs = _log_int(rng, 1, 256)
    hi = _log_int(rng, 16, max(64, 2000000 * 1024 // (seqs * hkv * d * 2)) if seqs > 8 else 65536)
    return dict(op=op, seqs=seqs, lo=rng.choice([1, max(1, hi // 2)]), hi=hi,
                take=_log_int(rng, 1, max(1, min(4096, 500000 // seqs) // page)), hq=hkv * rng.randint(1, 8), hkv=hkv,
                d=d, page=page, h=h, rot_v=rng.random() < 0.6, dt=dt, meta=meta)


# ----------------------------------------------------------------- helpers

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(seed, lo, hi, n):
    """n whole numbers in [lo, hi], on the CPU."""
    g = torch.Generator().manual_seed(int(seed) * 7 + 1)
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _chunk_bytes(c):
    return c["page"] * (c["d"] // 2 + 4)


def _summary_stride(c):
    """Bytes of a page's summary: every kv-head's codes, then every kv-head's word."""
    return (c["hkv"] * (c["d"] // 2 + 4) + 15) // 16 * 16


def _cache_views(cache, c):
    """A cache's packed codes [pages, hkv, page, d/2] and its metadata bytes [pages, hkv, page, 4]."""
    p, d = c["page"], c["d"]
    x = cache.view(-1, c["hkv"], _chunk_bytes(c))
    return x[:, :, :p * d // 2].unflatten(2, (p, d // 2)), x[:, :, p * d // 2:].unflatten(2, (p, 4))


def _summary_views(summary, c):
    """The summaries' packed codes [pages, hkv, d/2] and their metadata bytes [pages, hkv, 4]."""
    x, n = summary.view(-1, _summary_stride(c)), c["hkv"] * c["d"] // 2
    return x[:, :n].unflatten(1, (c["hkv"], c["d"] // 2)), x[:, n:n + 4 * c["hkv"]].unflatten(1, (c["hkv"], 4))


def _hadamard(x, h):
    """The block-diagonal Sylvester butterfly, ascending strides, then one product with 1/sqrt(h);
    each step one rounding in 32 bits, so the result is fixed to the bit."""
    shape, s = x.shape, 1
    while s < h:
        y = x.reshape(*shape[:-1], shape[-1] // (2 * s), 2, s)
        a, b = y[..., 0, :], y[..., 1, :]
        x = torch.stack((a + b, a - b), dim=-2).reshape(shape)
        s *= 2
    return x * float(np.float32(1.0 / math.sqrt(h)))


def _round_f16(x, up):
    """binary32 -> binary16 bits (int16), rounded up or down, saturating, a zero stored as +0."""
    x = x.clamp(-65504.0, 65504.0)
    h = x.half()
    b = h.view(torch.int16).to(torch.int32)
    b = torch.where(b < 0, -(b & 0x7FFF), b)            # ordered: +-0 are both 0
    f = h.float()
    b = b + (f < x).int() if up else b - (f > x).int()
    b = torch.where(b < 0, (-b) | 0x8000, b)
    return torch.where(b > 0x7FFF, b - 0x10000, b).to(torch.int16)


def _round_bf16(x, up):
    """The same to bfloat16 bits."""
    top = float(torch.finfo(torch.bfloat16).max)
    x = x.clamp(-top, top)
    w = x.contiguous().view(torch.int32)
    mag, neg = w & 0x7FFFFFFF, w < 0
    t = mag >> 16
    away = ((mag & 0xFFFF) != 0) & (~neg if up else neg)
    t = t + away.int()
    b = torch.where(neg & (t > 0), t | 0x8000, t)
    return torch.where(b > 0x7FFF, b - 0x10000, b).to(torch.int16)


def _quantize(x, c):
    """Rows float32 [..., d] -> packed codes uint8 [..., d/2] and {scale, zero} bytes uint8 [..., 4]."""
    mn, mx = x.amin(-1), x.amax(-1)
    if c["meta"] == "f16":
        z = _round_f16(mn, False)
        zf = z.view(torch.float16).float()
        s = _round_f16((mx - zf) / torch.full_like(mx, 15.0), True)
        sf = s.view(torch.float16).float()
    else:
        z = _round_bf16(mn, False)
        zf = z.view(torch.bfloat16).float()
        step = (mx - zf) / torch.full_like(mx, 15.0)
        s = _round_bf16(step, True)
        s = torch.where((step > 0) & (s < 0x80), torch.full_like(s, 0x80), s)
        sf = s.view(torch.bfloat16).float()
    r = torch.where(sf == 0, torch.zeros_like(sf), torch.ones_like(sf) / sf)
    q = torch.round((x - zf[..., None]) * r[..., None]).clamp(0, 15).to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), torch.stack((s, z), -1).view(torch.uint8)


def _append(x, slots, cache, c, rotate):
    """Rotate, quantize and scatter the rows x (float32 [T, hkv, d]) into a cache."""
    keep = slots >= 0
    x, slots = x[keep], slots[keep].long()
    q, m = _quantize(_hadamard(x, c["h"]) if rotate else x, c)
    codes, meta = _cache_views(cache, c)
    codes[slots // c["page"], :, slots % c["page"]] = q
    meta[slots // c["page"], :, slots % c["page"]] = m


def _codes(q):
    """Packed codes [..., n] -> float32 [..., 2 n]."""
    return torch.stack((q & 15, q >> 4), -1).flatten(-2).float()


def _words(m, c):
    """Metadata bytes [..., 4] -> scale and zero in float32."""
    m = m.contiguous().view(_DT[c["meta"]]).float()
    return m[..., 0], m[..., 1]


def _tables(c, seed, lens):
    """Shuffled block tables [seqs, blocks] of these lengths (-1 past a sequence's pages), and the pool's pages."""
    p, n = c["page"], len(lens)
    need = (lens + p - 1) // p
    pages = n * ((c["hi"] + p - 1) // p) + 4
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    e = torch.arange(int(need.max()))
    at = (need.cumsum(0) - need)[:, None] + e
    return torch.where(e < need[:, None], order[at.clamp(max=pages - 1)], torch.full((n, len(e)), -1)), pages


def _filled(c, gen, pages, rotate):
    """A cache of `pages` pages: heavy tails and a few outlier channels, a million rows at a time."""
    p, d, hkv = c["page"], c["d"], c["hkv"]
    cache = torch.zeros(pages * hkv * _chunk_bytes(c), dtype=torch.uint8, device="cuda")
    hot = torch.randint(0, d, (4,), generator=gen, device="cuda")
    run = max(p, (1 << 20) // hkv)
    for at in range(0, pages * p, run):
        slots = torch.arange(at, min(at + run, pages * p), device="cuda")
        x = torch.randn(len(slots), hkv, d, generator=gen, device="cuda")
        x *= torch.rand(len(slots), 1, 1, generator=gen, device="cuda") + 0.5
        x[:, :, hot] *= 8.0
        _append(x, slots, cache, c, rotate)
    return cache


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    c = dict(case)
    return {"norm_rope": _prep_norm_rope, "summary": _prep_summary, "select": _prep_select,
            "sparse": _prep_sparse}[c["op"]](c, seed)


def _status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def _prep_norm_rope(c, seed):
    t, hq, hkv, d, p = c["tokens"], c["hq"], c["hkv"], c["d"], c["page"]
    g = _gen(seed)
    # the projection's output: q, k and v side by side, a few outlier channels in k and v
    qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=g, device="cuda")
    hot = torch.randint(0, 2 * hkv * d, (8,), generator=g, device="cuda")
    qkv[:, hq * d + hot] *= 12.0
    qkv = qkv.to(_DT[c["dt"]])
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    pages = (t + p - 1) // p + 4
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    if c["chunk"]:                                       # one sequence's next tokens
        slots = order[i // p] * p + i % p
        pos = i + int(_ints(seed, 0, c["max_pos"] - t, 1))
    else:                                                # one token of each of t requests
        slots = torch.randperm(pages * p, generator=g, device="cuda")[:t]
        pos = torch.randint(0, c["max_pos"], (t,), generator=g, device="cuda")
        if t >= 64:
            slots[-t // 16:] = -1                        # the batch's padding
    # learned gains around 1, a few large ones, as w or as 1 + w
    w = 1.0 + 0.3 * torch.randn(2, d, generator=g, device="cuda")
    w[:, torch.randint(0, d, (2,), generator=g, device="cuda")] *= 4.0
    w = (w - c["offset"]).to(torch.float32 if c["wdt"] == "f32" else q.dtype)
    r = c["rope_dim"]
    a = torch.arange(c["max_pos"], device="cuda", dtype=torch.float64)[:, None] * torch.from_numpy(
        1e6 ** (-2.0 * np.arange(r // 2) / r)).cuda()
    n = pages * hkv * _chunk_bytes(c)
    return dict(c=c, q=q, k=k, v=v, wq=w[0], wk=w[1], pages=pages, slots=slots.int(), pos=pos.int(),
                cos_sin=torch.cat((a.cos(), a.sin()), 1).float(),
                q_out=torch.empty(t, hq, d, dtype=q.dtype, device="cuda"),
                kc=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                vc=torch.zeros(n, dtype=torch.uint8, device="cuda"), status=_status())


def _summary_lens(c, seed):
    lens = _ints(seed, c["lo"], c["hi"], c["seqs"])
    new = torch.full_like(lens, 1) if c["new"] == 1 else _ints(seed + 1, 1, c["new"], c["seqs"])
    if c["new"] >= c["hi"]:
        new = lens.clone()                               # whole prompts
    return lens, torch.minimum(new, lens)


def _prep_summary(c, seed):
    lens, new = _summary_lens(c, seed)
    bt, pages = _tables(c, seed, lens)
    return dict(c=c, pages=pages, kc=_filled(dict(c, h=min(128, c["d"])), _gen(seed), pages, True), bt=bt.int().cuda(),
                lens=lens.int().cuda(), new=new.int().cuda(), max_new=int(new.max()),
                summary=torch.zeros(pages * _summary_stride(c), dtype=torch.uint8, device="cuda"), status=_status())


def _prep_select(c, seed):
    lens = _ints(seed, c["lo"], c["hi"], c["seqs"])
    bt, pages = _tables(c, seed, lens)
    g = _gen(seed)
    b, hq, hkv, d = c["seqs"], c["hq"], c["hkv"], c["d"]
    # mean keys in the rotated domain: a bias that all pages share, each page's own part
    x = 0.4 * torch.randn(pages, hkv, d, generator=g, device="cuda")
    x += torch.randn(hkv, d, generator=g, device="cuda")
    summary = torch.zeros(pages * _summary_stride(c), dtype=torch.uint8, device="cuda")
    codes, meta = _summary_views(summary, c)
    codes[:], meta[:] = _quantize(x, c)
    del x
    shape = (b, hkv, c["take"])
    return dict(c=c, pages=pages, summary=summary, bt=bt.int().cuda(), lens=lens.int().cuda(), max_len=int(lens.max()),
                q=(torch.randn(b, hq, d, generator=g, device="cuda") * 2.0).to(_DT[c["dt"]]),
                tables=torch.empty(shape, dtype=torch.int32, device="cuda"),
                pages_out=torch.empty(shape, dtype=torch.int32, device="cuda"),
                sel_lens=torch.empty(b, hkv, dtype=torch.int32, device="cuda"), status=_status())


def _prep_sparse(c, seed):
    b, hq, hkv, d, p = c["seqs"], c["hq"], c["hkv"], c["d"], c["page"]
    lens = _ints(seed, c["lo"], c["hi"], b)
    bt, pages = _tables(c, seed, lens)
    g = _gen(seed)
    kc, vc = _filled(c, g, pages, True), _filled(c, g, pages, c["rot_v"])
    # every kv-head's own pages: the first, the last, others at random; ascending
    need, e = ((lens + p - 1) // p).cuda(), torch.arange(bt.shape[1], device="cuda")
    rank = torch.rand(b, hkv, len(e), generator=g, device="cuda")
    rank[:, :, 0] = -1.0
    rank.scatter_(2, (need - 1)[:, None, None].expand(b, hkv, 1), -2.0)
    rank = torch.where(e < need[:, None, None], rank, 2.0)
    k = min(c["take"], len(e))
    got, idx = rank.sort(-1)
    idx = torch.where(got[..., :k] < 2.0, idx[..., :k], len(e)).sort(-1)[0]
    pages_of = torch.cat((bt.cuda(), torch.full((b, 1), -1, device="cuda")), 1)
    tables = torch.gather(pages_of[:, None].expand(b, hkv, len(e) + 1), 2, idx)
    count = (idx < len(e)).sum(-1)
    sel_lens = (count - 1) * p + (lens.cuda() - (need - 1) * p)[:, None]
    return dict(c=c, pages=pages, kc=kc, vc=vc, tables=tables.int().contiguous(), sel_lens=sel_lens.int().contiguous(),
                max_len=int(sel_lens.max()), q=torch.randn(b, hq, d, generator=g, device="cuda").to(_DT[c["dt"]]),
                out=torch.empty(b, hq, d, dtype=_DT[c["dt"]], device="cuda"), status=_status())


# ----------------------------------------------------------------- run

def run(s):
    return {"norm_rope": _run_norm_rope, "summary": _run_summary, "select": _run_select,
            "sparse": _run_sparse}[s["c"]["op"]](s)


def _turn(x, c_, s_, inter):
    """x float32 [T, H, d]: its first 2 * pairs dims turned, each step one rounding."""
    n = c_.shape[-1]
    c_, s_ = c_[:, None], s_[:, None]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    y, z = a * c_ - b * s_, b * c_ + a * s_
    turned = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _norm(x, w, offset):
    """RMS norm of float32 rows; the squares are added neighbour by neighbour (a binary tree), each
    step one rounding, so the result is fixed to the bit."""
    t = x * x
    while t.shape[-1] > 1:
        t = t[..., 0::2] + t[..., 1::2]
    r = torch.ones_like(t) / torch.sqrt(t * (1.0 / x.shape[-1]) + float(np.float32(1e-6)))
    return x * r * (w.float() + offset)


def _run_norm_rope(s):
    c = s["c"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["pos"], s["cos_sin"], s["slots"],
                                 s["q_out"], s["kc"], s["vc"], s["pages"], c["page"], True, c["rot_v"], c["h"],
                                 eps=1e-6, weight_offset=c["offset"], interleaved=c["inter"], dev_status=s["status"],
                                 meta_bf16=c["meta"] == "bf16")
        return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
    cs = s["cos_sin"][s["pos"].long()]
    n = c["rope_dim"] // 2
    q = _turn(_norm(s["q"].float(), s["wq"], c["offset"]), cs[:, :n], cs[:, n:], c["inter"]).to(s["q"].dtype)
    k = _turn(_norm(s["k"].float(), s["wk"], c["offset"]), cs[:, :n], cs[:, n:], c["inter"])
    _append(k, s["slots"], s["kc"], c, True)
    _append(s["v"].float(), s["slots"], s["vc"], c, c["rot_v"])
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _run_summary(s):
    c, p = s["c"], s["c"]["page"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_page_summary(s["kc"], s["bt"], s["lens"], s["new"], s["max_new"], c["hkv"], c["d"], s["pages"], p,
                             s["summary"], dev_status=s["status"], meta_bf16=c["meta"] == "bf16")
        return {"summary": s["summary"]}
    e = torch.arange(s["bt"].shape[1], device="cuda")
    old, full = (s["lens"] - s["new"]) // p, s["lens"] // p
    pages = s["bt"][(e >= old[:, None]) & (e < full[:, None])].long()
    codes, meta = _cache_views(s["kc"], c)
    x, (sc, z) = codes[pages], _words(meta[pages], c)    # [n, hkv, p, d/2], [n, hkv, p]
    a, b = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    for t in range(0, p, 2):                             # even tokens and odd ones, in order
        a = a + _codes(x[:, :, t:t + 2]) * sc[:, :, t:t + 2, None]
        b = b + z[:, :, t:t + 2]
    a, b = a[:, :, 0] + a[:, :, 1], b[:, :, 0] + b[:, :, 1]
    q, m = _quantize((a + b[..., None]) * (1.0 / p), c)
    codes, meta = _summary_views(s["summary"], c)
    codes[pages], meta[pages] = q, m
    return {"summary": s["summary"]}


def _run_select(s):
    c, p = s["c"], s["c"]["page"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_select_pages(s["q"], s["summary"], s["bt"], s["lens"], s["max_len"], c["hkv"], s["pages"], p, True,
                             c["h"], c["first"], c["last"], s["tables"], s["sel_lens"], sel_pages=s["pages_out"],
                             dev_status=s["status"], meta_bf16=c["meta"] == "bf16")
        return {"tables": s["tables"], "pages": s["pages_out"], "lens": s["sel_lens"]}
    b, hq, hkv = c["seqs"], c["hq"], c["hkv"]
    # whole numbers -127 .. 127 for each q'
    q = _hadamard(s["q"].float(), c["h"])
    top = q.abs().amax(-1, keepdim=True)
    qs = top / torch.full_like(top, 127.0)
    r = torch.where(qs < 2.0 ** -126, torch.zeros_like(qs), torch.ones_like(qs) / qs)
    m = torch.round(q * r).clamp(-127, 127).view(b, hkv, hq // hkv, -1)
    codes, meta = _summary_views(s["summary"], c)
    ids = s["bt"].clamp(min=0).long()
    sc, z = (x.transpose(1, 2)[:, :, None] for x in _words(meta[ids], c))        # [b, hkv, 1, e]
    dot = torch.einsum("bhgd,behd->bhge", m, _codes(codes[ids]))                 # whole, below 2^24
    score = qs.view(b, hkv, -1, 1) * (sc * dot + z * m.sum(-1, keepdim=True))
    score = score.nan_to_num(nan=-math.inf, posinf=math.inf, neginf=-math.inf).amax(2)
    n = ((s["lens"] + p - 1) // p)[:, None, None]
    e = torch.arange(ids.shape[1], device="cuda")
    kind = torch.where((e < c["first"]) | (e >= n - c["last"]), 0, 1)
    kind = torch.where(e < n, kind, 2).expand_as(score)  # always taken; by score; not there
    idx = score.argsort(dim=-1, descending=True, stable=True)
    idx = idx.gather(-1, kind.gather(-1, idx).argsort(dim=-1, stable=True))[..., :c["take"]]
    idx = torch.where(kind.gather(-1, idx) < 2, idx, len(e)).sort(-1)[0]
    idx = torch.nn.functional.pad(idx, (0, c["take"] - idx.shape[-1]), value=len(e))
    there = idx < len(e)
    bt = torch.nn.functional.pad(s["bt"], (0, 1), value=-1)[:, None].expand(b, hkv, len(e) + 1)
    count = there.sum(-1)
    lens = torch.where(count > 0, count * p - (n * p - s["lens"][:, None, None])[..., 0], 0)
    return {"tables": bt.gather(-1, idx), "pages": torch.where(there, idx, -1).int(), "lens": lens.int()}


def _run_sparse(s):
    c, p = s["c"], s["c"]["page"]
    b, hq, hkv, d = c["seqs"], c["hq"], c["hkv"], c["d"]
    if own:
        import bit_paged_kv_gb300 as saw
        if "ws" not in s:                                # kept by the program, like its buffers
            need = saw.saw_sparse_decode_workspace_bytes(b, hq, hkv, d, p, s["max_len"])
            s["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
        saw.saw_sparse_decode_int4(s["q"], s["kc"], s["vc"], s["tables"], s["sel_lens"], s["max_len"], hkv, s["pages"],
                                   p, True, c["rot_v"], c["h"], s["out"], s["ws"], dev_status=s["status"],
                                   meta_bf16=c["meta"] == "bf16")
        return {"out": s["out"]}
    q = _hadamard(s["q"].float(), c["h"]).view(b, hkv, hq // hkv, d)
    at = (s["tables"].long().clamp(min=0), torch.arange(hkv, device="cuda")[:, None])

    def rows(cache):                                     # [b, hkv, tokens, d]
        codes, meta = _cache_views(cache, c)
        sc, z = _words(meta[at], c)
        return (_codes(codes[at]) * sc[..., None] + z[..., None]).flatten(2, 3)

    x = torch.einsum("bhgd,bhld->bhgl", q, rows(s["kc"])) / math.sqrt(d)
    x = x.masked_fill((torch.arange(x.shape[-1], device="cuda") >= s["sel_lens"][..., None])[:, :, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    o = torch.einsum("bhgl,bhld->bhgd", x, rows(s["vc"])) / x.sum(-1, keepdim=True)
    o = o.reshape(b, hq, d)
    return {"out": (_hadamard(o, c["h"]) if c["rot_v"] else o).to(s["q"].dtype)}


# ----------------------------------------------------------------- work

def work(case):
    c = case
    d, p, hkv = c["d"], c["page"], c["hkv"]
    row = d // 2 + 4                                     # a row of 4-bit values
    if c["op"] == "norm_rope":
        t, r = c["tokens"], c["rope_dim"]
        rows = t * hkv
        return {"bytes": t * c["hq"] * d * 4 + 2 * rows * (2 * d + row) + t * (4 * r + 8)
                + 2 * d * (4 if c["wdt"] == "f32" else 2),
                "flops": t * (c["hq"] + hkv) * (3 * r + 4 * d) + 2 * rows * d * (math.log2(c["h"]) + 6)}
    if c["op"] == "summary":
        lens, new = _summary_lens(c, 1)
        n = int((lens // p - (lens - new) // p).sum())
        return {"bytes": n * (hkv * (p + 1) * row + 4) + 8 * c["seqs"], "flops": 2 * n * hkv * p * d}
    if c["op"] == "select":
        n = (_ints(1, c["lo"], c["hi"], c["seqs"]) + p - 1) // p
        scored = int(torch.where(n > c["take"], n - c["first"] - c["last"], 0).sum())
        return {"bytes": scored * (hkv * row + 4) + c["seqs"] * (c["hq"] * d * 2 + 4 + hkv * (8 * c["take"] + 4)),
                "flops": 2 * scored * c["hq"] * d}
    lens = _ints(1, c["lo"], c["hi"], c["seqs"])
    n = (lens + p - 1) // p
    k = torch.minimum(n, torch.full_like(n, c["take"]))
    tokens = int((k * p - (n * p - lens)).sum())
    return {"bytes": hkv * (2 * tokens * row + 4 * int(k.sum()) + 4 * c["seqs"]) + c["seqs"] * c["hq"] * d * 4,
            "flops": 4 * d * c["hq"] * tokens}


# ----------------------------------------------------------------- exact

def exact(case, seed):
    """The computed numbers from their definitions, in 64 bits."""
    c = dict(case)
    if c["op"] in ("summary", "select"):
        return None                                      # whole numbers
    s = prepare(c, seed)
    d, hq, hkv, p, h = c["d"], c["hq"], c["hkv"], c["page"], None
    if c["op"] == "norm_rope":
        # the norm by the mean of the squares; each pair as a complex number times cos + i sin
        r, t = c["rope_dim"], c["tokens"]
        x = s["q"].double()
        out = x * torch.rsqrt(x.pow(2).mean(-1, keepdim=True) + 1e-6) * (s["wq"].double() + c["offset"])
        cs = s["cos_sin"].double()[s["pos"].long()]
        turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None]
        x = out[..., :r]
        pairs = x.reshape(t, -1, r // 2, 2) if c["inter"] else x.reshape(t, -1, 2, r // 2).transpose(2, 3)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        out[..., :r] = y.reshape(x.shape) if c["inter"] else y.transpose(2, 3).reshape(x.shape)
        return {"q": out, "k_cache": None, "v_cache": None}
    h = c["h"]
    m = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while m.shape[0] < h:
        m = torch.cat((torch.cat((m, m), 1), torch.cat((m, -m), 1)), 0)
    m = torch.block_diag(*[m / math.sqrt(h)] * (d // h))
    q = (s["q"].double() @ m).view(c["seqs"], hkv, hq // hkv, d)
    half = p * d // 2
    out = torch.zeros(c["seqs"], hkv, hq // hkv, d, dtype=torch.float64, device="cuda")
    lens = s["sel_lens"].tolist()
    for b in range(c["seqs"]):
        for head in range(hkv):
            n = lens[b][head]
            ids = s["tables"][b, head, :(n + p - 1) // p].long()
            rows = []
            for cache in (s["kc"], s["vc"]):
                x = cache.view(s["pages"], hkv, -1)[ids, head]               # [pages, chunk]
                code = x[:, :half].reshape(-1, d // 2)[:n]
                word = x[:, half:].reshape(-1, 4)[:n].contiguous().view(_DT[c["meta"]]).double()
                val = torch.empty(n, d, dtype=torch.float64, device="cuda")
                val[:, 0::2], val[:, 1::2] = (code & 15).double(), (code >> 4).double()
                rows.append(val * word[:, :1] + word[:, 1:])
            out[b, head] = torch.softmax(q[b, head] @ rows[0].T * d ** -0.5, dim=-1) @ rows[1]
    out = out.reshape(c["seqs"], hq, d)
    return {"out": out @ m if c["rot_v"] else out}
