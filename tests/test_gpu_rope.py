"""saw_rope_table and saw_rope_append.

The table against cosines and sines in 64 bits.  Its bound: the phase is cut
to 2^-32 turns (1.5e-9 rad), the angle within a quarter is rounded to
binary32 (half turns below 1/4: half a spacing is 2^-27 half turns, 2.4e-8
rad), sincospif is within 2 ulp (1.2e-7 below 1), the factor and the product
with it round once each (2^-24 together): 2.1e-7 < 2^-22 = 2.4e-7, times the
factor.

The append: the caches equal the rule byte for byte (binary32 rotary, each
operation rounded once, then the oracle's butterfly and directed rounding),
and q equals the rule's value rounded once to 16 bits; the rule itself is
checked against 64 bits: three roundings of 2^-24 and one of half a step.
"""
import math

import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
import oracle
from gpu_helpers import SENTINEL, assert_bytes_equal, bits, new_caches

pytestmark = pytest.mark.gpu


def freqs(r, base, kind, f=1.0, orig=0, low=0.0, high=0.0):
    """Radians per position of each pair and the factor, in Python floats."""
    out, att = [], 1.0
    b = base * f ** (r / (r - 2)) if kind == saw.SAW_ROPE_NTK else base
    if kind in (saw.SAW_ROPE_YARN, saw.SAW_ROPE_BANDS) and low == high == 0:
        low, high = 1.0, 32.0 if kind == saw.SAW_ROPE_YARN else 4.0
    for i in range(r // 2):
        w = b ** (-2 * i / r)
        if kind == saw.SAW_ROPE_LINEAR:
            w /= f
        if kind == saw.SAW_ROPE_BANDS:
            turns = orig * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            w = keep * w + (1 - keep) * w / f
        if kind == saw.SAW_ROPE_YARN:
            at = lambda t: r * math.log(orig / (2 * math.pi * t)) / (2 * math.log(base))
            lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), r - 1)
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w, att = w / f * ramp + w * (1 - ramp), 0.1 * math.log(f) + 1
        out.append(w)
    return np.array(out), att


@pytest.mark.parametrize("n,r,base,kind,f,orig,low,high", [
    (1, 16, 1e4, saw.SAW_ROPE_NONE, 1.0, 0, 0, 0),
    (131072, 128, 1e6, saw.SAW_ROPE_NONE, 1.0, 0, 0, 0),
    (1000, 256, 1e4, saw.SAW_ROPE_LINEAR, 8.0, 0, 0, 0),
    (777, 48, 5e5, saw.SAW_ROPE_NTK, 4.0, 0, 0, 0),
    (40000, 64, 1e6, saw.SAW_ROPE_YARN, 4.0, 8192, 0, 0),
    (5000, 112, 1e4, saw.SAW_ROPE_YARN, 2.0, 2048, 2.0, 16.0),
    (60000, 128, 5e5, saw.SAW_ROPE_BANDS, 8.0, 8192, 0, 0),
    (333, 96, 1e4, saw.SAW_ROPE_LINEAR, 0.1, 0, 0, 0),   # more than a turn per position
])
def test_table(n, r, base, kind, f, orig, low, high):
    t = torch.full((n + 1, r), 7.0, device="cuda")
    saw.saw_rope_table(t[:n], base, kind, f, orig, low, high)
    w, att = freqs(r, base, kind, f, orig, low, high)
    a = np.arange(n, dtype=np.float64)[:, None] * w
    want = att * np.concatenate((np.cos(a), np.sin(a)), 1)
    got = t[:n].cpu().numpy()
    # (the reference's own angle is off by a few 2^-53 of it)
    assert np.max(np.abs(got - want)) <= att * 2.0 ** -22 + 8 * 2.0 ** -53 * a.max()
    assert (t[n] == 7.0).all()


def test_table_explicit_factor():
    a, b = torch.empty(64, 64, device="cuda"), torch.empty(64, 64, device="cuda")
    saw.saw_rope_table(a, 1e4)
    saw.saw_rope_table(b, 1e4, att_scale=0.5)
    assert torch.equal(b, a * 0.5)


def turn(x, cs, r, inter, to=np.float32):
    """The rule on rows x [T, H, D] with table rows cs [T, r]; numpy rounds every operation once."""
    x = x.astype(to).copy()
    c, s = (v[:, None].astype(to) for v in (cs[:, :r // 2], cs[:, r // 2:]))
    a, b = (x[..., 0:r:2].copy(), x[..., 1:r:2].copy()) if inter else (x[..., :r // 2].copy(), x[..., r // 2:r].copy())
    y, z = a * c - b * s, b * c + a * s
    if inter:
        x[..., 0:r:2], x[..., 1:r:2] = y, z
    else:
        x[..., :r // 2], x[..., r // 2:r] = y, z
    return x


def oracle_cache(x, slots, pages, P, rotate, h, meta_bf16):
    """Quantize binary32 rows [T, H, D] by the append's rule into a sentinel-filled cache."""
    T, H, D = x.shape
    chunk = P * (D // 2 + 4)
    cache = np.full((pages, H, chunk), SENTINEL, np.uint8)
    y = oracle.rotate_canon(x, h) if rotate else x
    conv = oracle.f32_to_bf16_bits if meta_bf16 else oracle.f32_to_f16_bits
    val = (lambda b: (b.astype(np.uint32) << 16).view(np.float32)) if meta_bf16 else (lambda b: b.view(np.float16).astype(np.float32))
    z = conv(y.min(-1), oracle.RD)
    step = (y.max(-1) - val(z)) / np.float32(15)
    s = conv(step, oracle.RU)
    if meta_bf16:
        s = np.where((step > 0) & (s < 0x80), np.uint16(0x80), s)
    with np.errstate(divide="ignore"):
        r = np.where(val(s) == 0, np.float32(0), np.float32(1) / val(s))
    q = np.clip(np.rint((y - val(z)[..., None]) * r[..., None]), 0, 15).astype(np.uint8)
    q = q[..., 0::2] | (q[..., 1::2] << 4)
    words = np.stack((s, z), -1).astype(np.uint16).view(np.uint8)
    for t in range(T):
        if slots[t] >= 0:
            page, off = divmod(int(slots[t]), P)
            cache[page, :, off * D // 2:(off + 1) * D // 2] = q[t]
            cache[page, :, P * D // 2 + 4 * off:P * D // 2 + 4 * off + 4] = words[t]
    return cache.reshape(-1)


def make(seed, T, hq, hkv, D, P, r, dt, max_pos=40000, packed=True, spread=6.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device="cuda")
    x[:, torch.randint(0, x.shape[1], (5,), generator=g, device="cuda")] *= spread
    x = x.to(dt)
    q, k, v = (y.unflatten(1, (-1, D)) for y in x.split([hq * D, hkv * D, hkv * D], 1))
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pages = -(-T // P) + 3
    slots = torch.randperm(pages * P, generator=g, device="cuda")[:T].int()
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda").int()
    cs = torch.empty(max_pos, r, device="cuda")
    saw.saw_rope_table(cs, 1e4)
    return q, k, v, pages, slots, pos, cs


def run(q, k, v, pages, slots, pos, cs, P, rk, rv, h, inter, meta, q_out=None, stream=None):
    T, hkv, D = k.shape
    kc, vc = new_caches(pages, P, hkv, D, with_v=v is not None)
    if q is not None and q_out is None:
        q_out = torch.full(q.shape, -3.0, dtype=q.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    saw.saw_rope_append(q, k, v, pos, cs, slots, q_out, kc, vc, pages, P, rk, rv, h, interleaved=inter,
                        dev_status=st, meta_bf16=meta, stream=stream)
    torch.cuda.synchronize()
    return q_out, kc, vc, int(st.item())


def check(q, k, v, pages, slots, pos, cs, P, rk, rv, h, inter, meta, **kw):
    r, dt = cs.shape[1], k.dtype
    f32 = lambda x: x.float().cpu().numpy()
    q_in = None if q is None else f32(q)                 # (q_out may be q)
    qo, kc, vc, st = run(q, k, v, pages, slots, pos, cs, P, rk, rv, h, inter, meta, **kw)
    assert st == 0
    rows = cs[pos.long()].cpu().numpy()
    sl = slots.cpu().numpy()
    kr = turn(f32(k), rows, r, inter)
    assert_bytes_equal(kc, oracle_cache(kr, sl, pages, P, rk, h, meta), "K cache")
    if v is not None:
        assert_bytes_equal(vc, oracle_cache(f32(v), sl, pages, P, rv, h, meta), "V cache")
    if q is not None:
        y = turn(q_in, rows, r, inter)
        want = torch.from_numpy(y).to(dt)
        assert np.array_equal(bits(qo), bits(want))
        y64 = turn(q_in.astype(np.float64), rows, r, inter, np.float64)
        bound = np.abs(y64) * (torch.finfo(dt).eps / 2) + 3 * 2.0 ** -24 * 2 * np.abs(q_in).max() + torch.finfo(dt).tiny
        assert (np.abs(f32(qo) - y64) <= bound).all()
    return qo, kc, vc


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,r,h", [(64, 64, 64), (64, 16, 16), (64, 48, 32), (128, 128, 128), (128, 64, 64),
                                   (128, 16, 16), (128, 112, 128), (256, 256, 256), (256, 64, 32), (256, 208, 128)])
def test_head_dims_and_parts(D, r, h, inter):
    case = make(D + r, 37, 6, 2, D, 16, r, torch.bfloat16)
    check(*case, 16, True, True, h, inter, False)


@pytest.mark.parametrize("T,hq,hkv,P", [(1, 32, 8, 16), (2, 1, 1, 64), (255, 15, 3, 32), (600, 8, 8, 16),
                                        (1100, 32, 8, 64)])
@pytest.mark.parametrize("dt,meta", [(torch.bfloat16, False), (torch.float16, True)])
def test_sizes_and_formats(T, hq, hkv, P, dt, meta):
    case = make(T, T, hq, hkv, 128, P, 128, dt)
    check(*case, P, True, T % 2 == 0, 128, False, meta)


@pytest.mark.parametrize("rk,rv", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotations(rk, rv, D):
    case = make(9, 300, 4, 4, D, 16, D, torch.bfloat16, packed=False)
    check(*case, 16, bool(rk), bool(rv), 64, False, False)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [50, 2500])
def test_without_q_or_v_and_in_place(D, T):
    q, k, v, pages, slots, pos, cs = make(3, T, 4, 2, D, 16, D // 2, torch.bfloat16)
    check(None, k, v, pages, slots, pos, cs, 16, True, True, 64, False, False)
    check(q, k, None, pages, slots, pos, cs, 16, True, False, 64, True, False)
    check(q, k, v, pages, slots, pos, cs, 16, True, True, 64, False, False, q_out=q)


@pytest.mark.parametrize("D,hkv", [(128, 8), (128, 3), (64, 8), (64, 3), (256, 4), (256, 1)])
@pytest.mark.parametrize("inter", [False, True])
def test_bulk(D, hkv, inter):
    """Enough rows for the bulk kernel, an odd count, a part of the head and the whole of it."""
    T = 9001 // hkv
    for r, h, dt, meta in ((D, min(D, 128), torch.bfloat16, False), (D // 2, 32, torch.float16, True), (48, D, torch.bfloat16, True)):
        case = make(T + r, T, 2 * hkv, hkv, D, 16, r, dt)
        check(*case, 16, True, True, h, inter, meta)


@pytest.mark.parametrize("D,r", [(64, 16), (64, 32), (128, 16), (128, 32), (128, 64), (256, 16), (256, 64), (256, 128)])
@pytest.mark.parametrize("h", [16, 32, 64, 128])
def test_bulk_parts(D, r, h):
    """Turned parts whose pairs lie a power of two chunks apart, each with every block of the butterfly."""
    if h > D:
        h = 256 if D == 256 else D
    T = (5 << 18) // (13 * D) + 1
    case = make(D + r + h, T, 7, 3, D, 16, r, torch.bfloat16)
    check(*case, 16, True, h != 32, h, False, False)


@pytest.mark.parametrize("T", [64, 3000])
def test_padding_and_bad_entries(T):
    """Slot -1 appends nothing and turns q; a bad slot or position is skipped and reported."""
    q, k, v, pages, slots, pos, cs = make(5, T, 8, 4, 128, 16, 128, torch.bfloat16)
    slots[3] = slots[17] = slots[T - 1] = -1
    check(q, k, v, pages, slots, pos, cs, 16, True, True, 128, False, False)
    for what in ("slot", "slot_neg", "pos", "pos_neg"):
        s, p = slots.clone(), pos.clone()
        if what == "slot":
            s[9] = pages * 16
        elif what == "slot_neg":
            s[9] = -2
        elif what == "pos":
            p[9] = cs.shape[0]
        else:
            p[9] = -1
        qo, kc, vc, st = run(q, k, v, pages, s, p, cs, 16, True, True, 128, False, False)
        assert st == saw.SAW_ERR_DEVICE_INDEX
        ok = s.clone()
        ok[9] = -1
        rows = cs[pos.long()].cpu().numpy()
        f32 = lambda x: x.float().cpu().numpy()
        assert_bytes_equal(kc, oracle_cache(turn(f32(k), rows, 128, False), ok.cpu().numpy(), pages, 16, True, 128, False), what)
        assert_bytes_equal(vc, oracle_cache(f32(v), ok.cpu().numpy(), pages, 16, True, 128, False), what)
        want = bits(torch.from_numpy(turn(f32(q), rows, 128, False)).bfloat16()).copy()
        if "pos" in what:
            want[9] = bits(torch.full_like(q[9], -3.0))
        assert np.array_equal(bits(qo), want)


def test_position_zero_is_the_plain_append():
    """At position 0 nothing turns: the caches equal saw_quantize_append's."""
    q, k, v, pages, slots, pos, cs = make(8, 700, 8, 4, 128, 32, 128, torch.bfloat16, packed=False)
    qo, kc, vc, _ = run(q, k, v, pages, slots, torch.zeros_like(pos), cs, 32, True, True, 128, False, False)
    k2, v2 = new_caches(pages, 32, 4, 128)
    saw.saw_quantize_append(k, v, slots, k2, v2, pages, 32, True, True, 128)
    assert torch.equal(qo, q) and torch.equal(kc, k2) and torch.equal(vc, v2)


@pytest.mark.parametrize("T", [40, 4000])
def test_extreme_rows(T):
    """Constant, zero, huge and tiny rows; signed zeros; an outlier at a far position."""
    q, k, v, pages, slots, pos, cs = make(6, T, 2, 2, 128, 16, 128, torch.bfloat16)
    for i, val in enumerate((0.0, -0.0, 1.0, -3.0e4, 1e-30, 6.0e4)):
        k[i], v[i] = val, val
    k[7, :, 5], v[7, :, 5] = 5.0e4, -5.0e4
    for rk in (True, False):
        check(q, k, v, pages, slots, pos, cs, 16, rk, rk, 128, False, False)


@pytest.mark.parametrize("T", [64, 5000])
def test_other_stream_and_graph(T):
    q, k, v, pages, slots, pos, cs = make(4, T, 8, 2, 128, 16, 128, torch.bfloat16)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = run(q, k, v, pages, slots, pos, cs, 16, True, True, 128, False, False)
    b = run(q, k, v, pages, slots, pos, cs, 16, True, True, 128, False, False, stream=side)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    kc, vc = new_caches(pages, 16, 2, 128)
    qo = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_rope_append(q, k, v, pos, cs, slots, qo, kc, vc, pages, 16, True, True, 128)
    pos.copy_(pos.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    want = run(q, k, v, pages, slots, pos, cs, 16, True, True, 128, False, False)
    assert torch.equal(qo, want[0]) and torch.equal(kc, want[1]) and torch.equal(vc, want[2])
