"""Cases and plain forms of the serving-step operators around the INT4 paged cache.

Three operators and the table that one of them reads:

* ``tables``      block tables, slot mapping, positions and lengths of a batch, from cached
                  lengths, new-token counts and a list of free pages
* ``rope_table``  cosines and sines of every position, with the scalings for long contexts
* ``rope_append`` rotary positions on q and k, then the rotated, quantized append of k and v
* ``prefix``      decode attention of groups of sequences that share their first pages

``run`` computes the plain form with elementary torch operations, or with ``own`` set makes the
library's calls.  The caches come back as their bytes: the append's rule fixes every scale, zero
and code to the bit, so they are whole numbers that have to be equal.
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
        # a decode step of 64 running requests, 2048 to 16384 tokens each: rows of the pool's
        # table gathered by request, one new token per request
        dict(name="tables-decode-64", op="tables", seqs=64, lo=2048, hi=16384, new=1, page=16,
             gather=True, short=False),
        # 4096 requests up to 32768 tokens with chunks of up to 256 new tokens, page 16
        dict(name="tables-mixed-4096", op="tables", seqs=4096, lo=0, hi=32768, new=256, page=16,
             gather=True, short=False),
        # the table of a 32768-token model, whole head, no scaling
        dict(name="rope-table-32768", op="rope_table", max_pos=32768, rope_dim=128, base=1e6,
             scaling="none", factor=1.0, orig=0),
        # a context stretched four times to 131072 positions
        dict(name="rope-table-yarn-131072", op="rope_table", max_pos=131072, rope_dim=128,
             base=1e6, scaling="yarn", factor=4.0, orig=32768),
        # one decoding request at a far position: latency
        dict(name="rope-append-1", op="rope_append", tokens=1, hq=32, hkv=8, d=128, page=16,
             rope_dim=128, inter=False, h=128, rot_v=False, dt="bf16", meta="f16",
             max_pos=32768, chunk=False),
        # a decode step of 256 requests, padded rows among them, 64 q-heads
        dict(name="rope-append-256", op="rope_append", tokens=256, hq=64, hkv=8, d=128, page=16,
             rope_dim=128, inter=True, h=128, rot_v=True, dt="bf16", meta="f16",
             max_pos=32768, chunk=False),
        # an odd prefill chunk in binary16, half of each head turned, bfloat16 metadata
        dict(name="rope-append-2047-part", op="rope_append", tokens=2047, hq=32, hkv=8, d=128,
             page=32, rope_dim=64, inter=False, h=64, rot_v=True, dt="f16", meta="bf16",
             max_pos=32768, chunk=True),
        # the long prompt: 131072 tokens at once
        dict(name="rope-append-131072", op="rope_append", tokens=131072, hq=32, hkv=8, d=128,
             page=64, rope_dim=128, inter=False, h=128, rot_v=True, dt="bf16", meta="f16",
             max_pos=131072, chunk=True),
        # four answers sampled from one prompt: latency
        dict(name="prefix-4x1024", op="prefix", seqs=4, groups=1, prefix=1024, lo=1, hi=64, hq=32,
             hkv=8, page=16, rot_v=False, h=128, dt="bf16", meta="f16"),
        # 64 chats behind one 16384-token document
        dict(name="prefix-64x16384", op="prefix", seqs=64, groups=1, prefix=16384, lo=128, hi=2048,
             hq=32, hkv=8, page=16, rot_v=True, h=128, dt="bf16", meta="f16"),
        # 256 chats behind one 4096-token system prompt, 64 q-heads
        dict(name="prefix-256x4096", op="prefix", seqs=256, groups=1, prefix=4096, lo=64, hi=1024,
             hq=64, hkv=8, page=16, rot_v=True, h=128, dt="bf16", meta="f16"),
        # 37 requests behind five different prompts of odd lengths, one of them not shared
        dict(name="prefix-37-in-5", op="prefix", seqs=37, groups=5, prefix=24000, lo=1, hi=3000,
             hq=32, hkv=8, page=64, rot_v=True, h=64, dt="f16", meta="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "rope_table", "rope_append", "rope_append", "prefix", "prefix"])
    if op == "tables":
        lo = rng.choice([0, 1, 500, 2048])
        return dict(op=op, seqs=_log_int(rng, 1, 4096), lo=lo,
                    hi=lo + _log_int(rng, 16, 30000), new=rng.choice([1, 1, 17, 256]),
                    page=rng.choice([16, 32, 64]), gather=rng.random() < 0.5,
                    short=rng.random() < 0.3)
    if op == "rope_table":
        scaling = rng.choice(["none", "linear", "ntk", "yarn", "bands"])
        return dict(op=op, max_pos=_log_int(rng, 200, 131072), rope_dim=16 * rng.randint(2, 8),
                    base=rng.choice([1e4, 5e5, 1e6]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    orig=rng.choice([4096, 8192, 32768]))
    if op == "rope_append":
        d = rng.choice([64, 128, 128, 256])
        hkv = rng.choice([1, 2, 3, 4, 8])
        tokens = _log_int(rng, 1, max(2, min(60000, 60000 * 1024 // (hkv * d))))
        return dict(op=op, tokens=tokens, hq=hkv * rng.randint(1, 8 if tokens < 20000 else 4),
                    hkv=hkv, d=d, page=rng.choice([16, 32, 64]),
                    rope_dim=16 * rng.randint(1, d // 16) if rng.random() < 0.5 else d,
                    inter=rng.random() < 0.5, h=rng.choice([h for h in (16, 32, 64, 128, 256) if h <= d]),
                    rot_v=rng.random() < 0.6, dt=rng.choice(["bf16", "f16"]),
                    meta=rng.choice(["f16", "f16", "bf16"]), max_pos=rng.choice([32768, 131072]),
                    chunk=tokens > 512)
    seqs = _log_int(rng, 1, 256)
    prefix = _log_int(rng, 16, min(32768, 1000000 // seqs))
    hkv = rng.choice([1, 2, 4, 8])
    return dict(op=op, seqs=seqs, groups=rng.choice([1, 1, 2, 3, 7]) if seqs > 8 else 1,
                prefix=prefix, lo=1, hi=_log_int(rng, 2, 2048 if seqs < 128 else 1024),
                hq=hkv * rng.randint(1, 8), hkv=hkv, page=rng.choice([16, 32, 64]),
                rot_v=rng.random() < 0.6, h=rng.choice([64, 128]), dt=rng.choice(["bf16", "f16"]),
                meta=rng.choice(["f16", "f16", "bf16"]))


# ----------------------------------------------------------------- helpers

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _ints(seed, lo, hi, n):
    """n whole numbers in [lo, hi], on the CPU."""
    g = torch.Generator().manual_seed(int(seed) * 7 + 1)
    return torch.randint(lo, hi + 1, (n,), generator=g)


def _chunk_bytes(c):
    return c["page"] * (c.get("d", 128) // 2 + 4)


def _cache_views(cache, pages, c):
    """A cache's packed codes [pages, hkv, page, d/2] and its metadata bytes [pages, hkv, page, 4]."""
    p, d, hkv = c["page"], c.get("d", 128), c["hkv"]
    x = cache.view(pages, hkv, _chunk_bytes(c))
    return (x[:, :, :p * d // 2].unflatten(2, (p, d // 2)),
            x[:, :, p * d // 2:].unflatten(2, (p, 4)))


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
    w = x.view(torch.int32)
    mag, neg = w & 0x7FFFFFFF, w < 0
    t = mag >> 16
    away = ((mag & 0xFFFF) != 0) & (~neg if up else neg)
    t = t + away.int()
    b = torch.where(neg & (t > 0), t | 0x8000, t)
    return torch.where(b > 0x7FFF, b - 0x10000, b).to(torch.int16)


def _append(x, slots, cache, pages, c, rotate):
    """Rotate, quantize and scatter the rows x (float32 [T, hkv, d]) into a cache."""
    keep = slots >= 0
    x, slots = x[keep], slots[keep].long()
    if rotate:
        x = _hadamard(x, c["h"])
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
    q = q[..., 0::2] | (q[..., 1::2] << 4)
    codes, meta = _cache_views(cache, pages, c)
    page, off = slots // c["page"], slots % c["page"]
    codes[page, :, off] = q
    meta[page, :, off] = torch.stack((s, z), -1).view(torch.uint8)


def _values(cache, pages, c, page, off, to):
    """Dequantized rows [..., hkv, d] of the slots (page, off), in the cache's (rotated) domain."""
    codes, meta = _cache_views(cache, pages, c)
    q = codes[page, :, off]
    m = meta[page, :, off].contiguous().view(torch.float16 if c["meta"] == "f16" else torch.bfloat16).to(to)
    q = torch.stack((q & 15, q >> 4), -1).flatten(-2).to(to)
    return q * m[..., 0:1] + m[..., 1:2]


def _inv_freq(c):
    """Radians per position of every pair, and the factor on the cosines and sines; host, 64 bits."""
    r, base, f = c["rope_dim"], c["base"], c["factor"]
    i = np.arange(r // 2, dtype=np.float64)
    if c["scaling"] == "ntk" and r > 2:
        base = base * f ** (r / (r - 2))
    inv, att = base ** (-2.0 * i / r), 1.0
    if c["scaling"] == "linear":
        inv = inv / f
    elif c["scaling"] == "yarn":
        def dim(beta):
            return r * math.log(c["orig"] / (2 * math.pi * beta)) / (2 * math.log(base))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), r - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        inv, att = inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    elif c["scaling"] == "bands":
        turns = c["orig"] * inv / (2 * math.pi)          # turns within the original context
        smooth = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        inv = (1 - smooth) * inv / f + smooth * inv
    return inv, att


def _rope_cos_sin(c, device="cuda"):
    inv, att = _inv_freq(c)
    a = torch.arange(c["max_pos"], device=device, dtype=torch.float64)[:, None] * torch.from_numpy(inv).to(device)
    return torch.cat((a.cos(), a.sin()), 1) * att


# ----------------------------------------------------------------- prepare

def prepare(case, seed):
    c = dict(case)
    return {"tables": _prep_tables, "rope_table": _prep_rope_table, "rope_append": _prep_rope_append,
            "prefix": _prep_prefix}[c["op"]](c, seed)


def _prep_tables(c, seed):
    n, p = c["seqs"], c["page"]
    cached = _ints(seed, c["lo"], c["hi"], n)
    new = _ints(seed + 1, 1, c["new"], n)
    if n > 4:
        cached[n // 2] = 0                               # a request that begins
    old = (cached + p - 1) // p
    need = (cached + new + p - 1) // p - old
    blocks = (c["hi"] + c["new"] + p - 1) // p + 1
    rows = n + n // 8 + 1                                # the pool keeps rows of waiting requests
    pages = int(old.sum() + need.sum()) + 64
    ids = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    src_rows = torch.randperm(rows, generator=torch.Generator().manual_seed(seed + 1))[:n] if c["gather"] else torch.arange(n)
    src = torch.full((rows, blocks), -1, dtype=torch.int32)
    e = torch.arange(blocks)
    first = old.cumsum(0) - old
    own_pages = ids[(first[:, None] + e).clamp(max=pages - 1)]
    src[src_rows] = torch.where(e < old[:, None], own_pages, src[src_rows])
    free = ids[int(old.sum()):].contiguous()
    num_free = int(need.sum()) * 3 // 4 if c["short"] else free.numel()
    tokens = n * c["new"]                                # the largest step: the batch is padded
    dev = "cuda"
    s = dict(c=c, cached=cached.int().to(dev), new=new.int().to(dev), src=src.to(dev), free=free.to(dev),
             num_free=torch.tensor([num_free], dtype=torch.int32, device=dev), pages=pages,
             src_rows=src_rows.int().to(dev) if c["gather"] else None, seqs=n, blocks=blocks, tokens=tokens,
             status=torch.zeros(1, dtype=torch.int32, device=dev))
    s.update(bt=torch.full((n, blocks), -1, dtype=torch.int32, device=dev),
             lens=torch.empty(n, dtype=torch.int32, device=dev),
             cu=torch.empty(n + 1, dtype=torch.int32, device=dev),
             slots=torch.empty(tokens, dtype=torch.int32, device=dev),
             pos=torch.empty(tokens, dtype=torch.int32, device=dev),
             taken=torch.empty(1, dtype=torch.int32, device=dev))
    return s


def _prep_rope_table(c, seed):
    # another seed is another model: its base differs a little
    c["base"] = c["base"] * (1.0 + 1e-3 * (seed % 997))
    return dict(c=c, out=torch.empty(c["max_pos"], c["rope_dim"], dtype=torch.float32, device="cuda"))


def _prep_rope_append(c, seed):
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
    table = dict(rope_dim=c["rope_dim"], base=1e6, factor=1.0, scaling="none", max_pos=c["max_pos"])
    n = pages * hkv * _chunk_bytes(c)
    return dict(c=c, q=q, k=k, v=v, pages=pages, slots=slots.int(), pos=pos.int(),
                cos_sin=_rope_cos_sin(table).float(),
                q_out=torch.empty(t, hq, d, dtype=q.dtype, device="cuda"),
                kc=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                vc=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _groups(c, seed):
    """First sequence of each group, and each group's prefix length (whole pages)."""
    n, k, p = c["seqs"], c["groups"], c["page"]
    cuts = sorted(set(_ints(seed + 5, 1, n - 1, k - 1).tolist())) if k > 1 else []
    cu = [0] + cuts + [n]
    lens = [c["prefix"]] + _ints(seed + 6, 0, c["prefix"], len(cu) - 2).tolist()
    if len(lens) > 2:
        lens[1] = 0                                      # a group that shares nothing
    return cu, [x // p * p for x in lens]


def _prep_prefix(c, seed):
    n, p, hkv, hq, d = c["seqs"], c["page"], c["hkv"], c["hq"], 128
    cu, pre = _groups(c, seed)
    rest = _ints(seed, c["lo"], c["hi"], n)
    pre_of = torch.zeros(n, dtype=torch.int64)
    pages = sum(x // p for x in pre)
    order = torch.randperm(pages + int(((rest + p - 1) // p).sum()) + 4, generator=torch.Generator().manual_seed(seed))
    blocks = max(pre) // p + (c["hi"] + p - 1) // p
    bt = torch.full((n, blocks), -1, dtype=torch.int64)
    nxt = 0
    for g, x in enumerate(pre):
        bt[cu[g]:cu[g + 1], :x // p] = order[nxt:nxt + x // p]
        pre_of[cu[g]:cu[g + 1]] = x
        nxt += x // p
    for b in range(n):
        a, m = int(pre_of[b]) // p, (int(rest[b]) + p - 1) // p
        bt[b, a:a + m] = order[nxt:nxt + m]
        nxt += m
    pages = order.numel()
    gen = _gen(seed)
    size = pages * hkv * _chunk_bytes(c)
    caches = []
    for rotate in (True, c["rot_v"]):                    # heavy tails and a few outlier channels
        x = torch.randn(pages * p, hkv, d, generator=gen, device="cuda")
        x *= torch.rand(pages * p, 1, 1, generator=gen, device="cuda") + 0.5
        x[:, :, torch.randint(0, d, (4,), generator=gen, device="cuda")] *= 8.0
        cache = torch.zeros(size, dtype=torch.uint8, device="cuda")
        _append(x, torch.arange(pages * p, device="cuda"), cache, pages, c, rotate)
        caches.append(cache)
        del x
    s = dict(c=c, kc=caches[0], vc=caches[1], pages=pages, cu_h=cu, pre_h=pre,
             q=torch.randn(n, hq, d, generator=gen, device="cuda").to(_DT[c["dt"]]),
             bt=bt.int().cuda(), lens=(pre_of + rest).int().cuda(),
             cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             pre=torch.tensor(pre, dtype=torch.int32, device="cuda"),
             status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    s["out"] = torch.empty_like(s["q"])
    s["max_pre"], s["max_rest"] = max(pre), int(rest.max())
    if own:
        import bit_paged_kv_gb300 as saw
        need = saw.saw_prefix_decode_workspace_bytes(n, len(pre), hq, hkv, d, p, s["max_pre"], s["max_rest"])
        s["ws"] = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    return s


# ----------------------------------------------------------------- run

def run(s):
    return {"tables": _run_tables, "rope_table": _run_rope_table, "rope_append": _run_rope_append,
            "prefix": _run_prefix}[s["c"]["op"]](s)


def _run_tables(s):
    c, p = s["c"], s["c"]["page"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_build_tables(s["cached"], s["new"], s["free"], s["num_free"], p, s["pages"], s["bt"],
                             s["lens"], s["cu"], s["slots"], s["pos"], s["taken"], src_tables=s["src"],
                             src_rows=s["src_rows"], dev_status=s["status"])
        return {k: s[k] for k in ("bt", "lens", "cu", "slots", "pos", "taken")}
    cached, new, n = s["cached"].long(), s["new"].long(), s["seqs"]
    old = (cached + p - 1) // p
    need = (cached + new + p - 1) // p - old
    off = need.cumsum(0) - need
    end = off + need
    fits = (need == 0) | (end <= s["num_free"])          # one that needs no page is always served
    taken = torch.where(end <= s["num_free"], end, torch.zeros_like(end)).amax().reshape(1)
    cu = torch.cat((torch.zeros_like(new[:1]), new.cumsum(0)))
    src = s["src"][s["src_rows"].long()] if s["src_rows"] is not None else s["src"][:n]
    e = torch.arange(s["blocks"], device="cuda")
    fresh = s["free"][(off[:, None] + e - old[:, None]).clamp(0, s["free"].numel() - 1)]
    bt = torch.where(e < old[:, None], src, torch.where((e < (old + need)[:, None]) & fits[:, None], fresh, s["bt"]))
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    pos = cached[b] + t - cu[b]
    real = t < cu[-1]
    page = bt[b, (pos // p).clamp(0, s["blocks"] - 1)].long()
    slots = torch.where(real & fits[b], page * p + pos % p, -1)
    lens = torch.where(fits, cached + new, cached)
    return {"bt": bt, "lens": lens.int(), "cu": cu.int(), "slots": slots.int(),
            "pos": torch.where(real & fits[b], pos, 0).int(), "taken": taken.int()}


def _run_rope_table(s):
    c = s["c"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_rope_table(s["out"], base=c["base"], scaling=getattr(saw, "SAW_ROPE_" + c["scaling"].upper()),
                           factor=c["factor"], orig_max_pos=c["orig"])
        return {"cos_sin": s["out"]}
    return {"cos_sin": _rope_cos_sin(c).float()}


def _turn(x, c_, s_, inter):
    """x float32 [T, H, d]: its first 2 * pairs dims turned, each step one rounding."""
    n = c_.shape[-1]
    c_, s_ = c_[:, None], s_[:, None]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if inter else (x[..., :n], x[..., n:2 * n])
    y, z = a * c_ - b * s_, b * c_ + a * s_
    turned = torch.stack((y, z), -1).flatten(-2) if inter else torch.cat((y, z), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _run_rope_append(s):
    c = s["c"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_rope_append(s["q"], s["k"], s["v"], s["pos"], s["cos_sin"], s["slots"], s["q_out"], s["kc"],
                            s["vc"], s["pages"], c["page"], True, c["rot_v"], c["h"], interleaved=c["inter"],
                            dev_status=s["status"], meta_bf16=c["meta"] == "bf16")
        return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
    cs = s["cos_sin"][s["pos"].long()]
    n = c["rope_dim"] // 2
    q = _turn(s["q"].float(), cs[:, :n], cs[:, n:], c["inter"]).to(s["q"].dtype)
    _append(_turn(s["k"].float(), cs[:, :n], cs[:, n:], c["inter"]), s["slots"], s["kc"], s["pages"], c, True)
    _append(s["v"].float(), s["slots"], s["vc"], s["pages"], c, c["rot_v"])
    return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}


def _run_prefix(s):
    c = s["c"]
    p, hkv, hq = c["page"], c["hkv"], c["hq"]
    if own:
        import bit_paged_kv_gb300 as saw
        saw.saw_prefix_decode_int4(s["q"], s["kc"], s["vc"], s["bt"], s["lens"], s["cu"], s["pre"], s["max_pre"],
                                   s["max_rest"], hkv, s["pages"], p, True, c["rot_v"], c["h"], s["out"], s["ws"],
                                   dev_status=s["status"], meta_bf16=c["meta"] == "bf16")
        return {"out": s["out"]}
    n = s["q"].shape[0]
    q = _hadamard(s["q"].float(), c["h"]).view(n, hkv, hq // hkv, 128)
    t = torch.arange(int(s["lens"].max()), device="cuda")
    page = s["bt"].long().clamp(min=0)[:, t // p]        # [n, L]; a sequence's own pages, prefix first
    off = (t % p).expand_as(page)
    k = _values(s["kc"], s["pages"], c, page, off, torch.float32)
    x = torch.einsum("nhgd,nlhd->nhgl", q, k) / math.sqrt(128.0)
    del k
    x = x.masked_fill((t >= s["lens"][:, None])[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    v = _values(s["vc"], s["pages"], c, page, off, torch.float32)
    o = torch.einsum("nhgl,nlhd->nhgd", x, v) / x.sum(-1, keepdim=True)
    o = o.reshape(n, hq, 128)
    return {"out": (_hadamard(o, c["h"]) if c["rot_v"] else o).to(s["q"].dtype)}


# ----------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "tables":
        s = _prep_sizes(c)
        # the gathered entries in and out, the taken pages, per-request words, slots and positions
        return {"bytes": 8 * s["old"] + 8 * s["need"] + 24 * c["seqs"] + 8 * c["seqs"] * c["new"], "flops": 0}
    if c["op"] == "rope_table":
        return {"bytes": 4 * c["max_pos"] * c["rope_dim"], "flops": c["max_pos"] * c["rope_dim"]}
    if c["op"] == "rope_append":
        t, d, r = c["tokens"], c["d"], c["rope_dim"]
        rows = t * c["hkv"]
        return {"bytes": t * c["hq"] * d * 4 + 2 * rows * (2 * d + d // 2 + 4) + t * (4 * r + 8),
                "flops": t * (c["hq"] + c["hkv"]) * 3 * r + 2 * rows * d * (math.log2(c["h"]) + 6)}
    cu, pre = _groups(c, 1)
    rest = int(_ints(1, c["lo"], c["hi"], c["seqs"]).sum())
    row = 2 * c["hkv"] * (64 + 4)
    seen = sum(x * (cu[g + 1] - cu[g]) for g, x in enumerate(pre)) + rest
    return {"bytes": row * (sum(pre) + rest) + c["seqs"] * c["hq"] * 128 * 4 + 4 * seen // c["page"],
            "flops": 4 * 128 * c["hq"] * seen}


def _prep_sizes(c):
    n, p = c["seqs"], c["page"]
    cached, new = _ints(1, c["lo"], c["hi"], n), _ints(2, 1, c["new"], n)
    old = (cached + p - 1) // p
    return dict(old=int(old.sum()), need=int(((cached + new + p - 1) // p - old).sum()))


# ----------------------------------------------------------------- exact

def _one_freq(c, i):
    """Radians per position of pair i, pair by pair."""
    r, f = c["rope_dim"], c["factor"]
    plain = math.exp(-2 * i / r * math.log(c["base"]))
    if c["scaling"] == "none":
        return plain
    if c["scaling"] == "linear":
        return plain / f
    if c["scaling"] == "ntk":
        return math.exp(-2 * i / r * (math.log(c["base"]) + r / (r - 2) * math.log(f)))
    if c["scaling"] == "bands":
        wave = 2 * math.pi / plain                       # positions per turn
        if wave > c["orig"] / 1.0:
            return plain / f
        if wave < c["orig"] / 4.0:
            return plain
        mix = (c["orig"] / wave - 1.0) / (4.0 - 1.0)
        return mix * plain + (1 - mix) * plain / f
    # yarn: the pairs that turn 32 times and once within the original context bound the ramp
    at = [r / 2 * math.log(c["orig"] / (2 * math.pi * turns)) / math.log(c["base"]) for turns in (32, 1)]
    first, last = max(0, math.floor(at[0])), min(r - 1, math.ceil(at[1]))
    share = min(1.0, max(0.0, (i - first) / max(last - first, 0.001)))
    return plain * (share / f + 1 - share)


def exact(case, seed):
    """The operators' computed numbers from their definitions, in 64 bits."""
    c = dict(case)
    if c["op"] == "tables":
        return None
    s = prepare(c, seed)
    if c["op"] == "rope_table":
        c = s["c"]
        freq = torch.tensor([_one_freq(c, i) for i in range(c["rope_dim"] // 2)], dtype=torch.float64)
        a = torch.outer(torch.arange(c["max_pos"], dtype=torch.float64), freq).cuda()
        grow = 1.0 + 0.1 * math.log(c["factor"]) if c["scaling"] == "yarn" else 1.0
        return {"cos_sin": torch.cat((grow * torch.cos(a), grow * torch.sin(a)), dim=-1)}
    if c["op"] == "rope_append":
        # each pair as a complex number times cos + i sin
        r, t = c["rope_dim"], c["tokens"]
        cs = s["cos_sin"].double()[s["pos"].long()]
        turn = torch.complex(cs[:, :r // 2], cs[:, r // 2:])[:, None]
        out = s["q"].double()
        x = out[..., :r]
        pairs = x.reshape(t, -1, r // 2, 2) if c["inter"] else x.reshape(t, -1, 2, r // 2).transpose(2, 3)
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        out[..., :r] = y.reshape(x.shape) if c["inter"] else y.transpose(2, 3).reshape(x.shape)
        return {"q": out, "k_cache": None, "v_cache": None}
    n, hq, hkv, p, h = c["seqs"], c["hq"], c["hkv"], c["page"], c["h"]
    m = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while m.shape[0] < h:
        m = torch.cat((torch.cat((m, m), 1), torch.cat((m, -m), 1)), 0)
    m = torch.block_diag(*[m / math.sqrt(h)] * (128 // h))
    q = (s["q"].double() @ m).view(n, hkv, hq // hkv, 128)
    outs = []
    for b in range(n):
        t = torch.arange(int(s["lens"][b]), device="cuda")
        page, off = s["bt"][b].long()[t // p], t % p
        rows = []
        for cache in (s["kc"], s["vc"]):
            x = cache.view(s["pages"], hkv, -1)[page]                # [L, hkv, chunk]
            code = x[:, :, :p * 64].view(-1, hkv, p, 64)[torch.arange(len(t)), :, off]
            word = x[:, :, p * 64:].contiguous().view(torch.int16).view(-1, hkv, p, 2)[torch.arange(len(t)), :, off]
            word = word.contiguous().view(_DT[c["meta"]]).double()
            val = torch.empty(len(t), hkv, 128, dtype=torch.float64, device="cuda")
            val[..., 0::2], val[..., 1::2] = (code & 15).double(), (code >> 4).double()
            rows.append(val * word[..., :1] + word[..., 1:])
        w = torch.softmax(torch.einsum("hgd,lhd->hgl", q[b], rows[0]) * 128 ** -0.5, dim=-1)
        outs.append(torch.einsum("hgl,lhd->hgd", w, rows[1]).reshape(hq, 128))
    o = torch.stack(outs)
    return {"out": o @ m if c["rot_v"] else o}
