"""saw_norm_rope_append: the caches equal the rule byte for byte (the norm and the
rotary turn in binary32, each operation rounded once, then the append's
quantizer), q equals the rule's value rounded once to 16 bits, and the rule is
checked against 64 bits.

With u = 2^-24: the sum of squares is off by log2 D + 1 <= 9 roundings, halved
by the root; the mean and eps add two before the root, halved too; root,
reciprocal, product with r, gain and product with it are one each: 10.5 u.  The
turn of a pair adds 2 u to each product and one more to their sum, on values of
at most sqrt 2 times the row's largest: 16 u times twice that holds.  Then one
rounding to 16 bits.
"""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from gpu_helpers import assert_bytes_equal, bits, new_caches
from sparse_oracle import U, norm_rows
from test_gpu_rope import make, oracle_cache, turn

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def gains(D, dt, offset, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = 1 + 0.3 * torch.randn(2, D, generator=g, device="cuda")
    w[:, 3] *= 5
    return (w - offset).to(dt)


def run(q, k, v, wq, wk, pages, slots, pos, cs, P, rk, rv, h, inter=False, meta=False, eps=1e-6, offset=0.0, q_out=None,
        stream=None):
    T, hkv, D = k.shape
    kc, vc = new_caches(pages, P, hkv, D, with_v=v is not None)
    if q is not None and q_out is None:
        q_out = torch.full(q.shape, -3.0, dtype=q.dtype, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    saw.saw_norm_rope_append(q, k, v, wq, wk, pos, cs, slots, q_out, kc, vc, pages, P, rk, rv, h, eps=eps,
                             weight_offset=offset, interleaved=inter, dev_status=st, meta_bf16=meta, stream=stream)
    torch.cuda.synchronize()
    return q_out, kc, vc, int(st.item())


def f32(x):
    return None if x is None else x.float().cpu().numpy()


def check(q, k, v, pages, slots, pos, cs, P, rk, rv, h, inter, meta, w=(None, None), eps=1e-6, offset=0.0, status=0,
          skip=(), **kw):
    r, dt = cs.shape[1], k.dtype
    q_in = f32(q)                                        # (q_out may be q)
    qo, kc, vc, st = run(q, k, v, *w, pages, slots, pos, cs, P, rk, rv, h, inter, meta, eps, offset, **kw)
    assert st == status
    rows = cs[pos.long().clamp(0, cs.shape[0] - 1)].cpu().numpy()
    sl = slots.cpu().numpy().copy()
    sl[(sl < 0) | (sl >= pages * P)] = -1
    sl[list(skip)] = -1
    kr = turn(norm_rows(f32(k), f32(w[1]), offset, eps), rows, r, inter)
    assert_bytes_equal(kc, oracle_cache(kr, sl, pages, P, rk, h, meta), "K cache")
    if v is not None:
        assert_bytes_equal(vc, oracle_cache(f32(v), sl, pages, P, rv, h, meta), "V cache")
    if q is not None:
        y = norm_rows(q_in, f32(w[0]), offset, eps)
        want = bits(torch.from_numpy(turn(y, rows, r, inter)).to(dt)).copy()
        for t in skip:
            want[t] = bits(torch.full_like(q[t], -3.0))
        assert np.array_equal(bits(qo), want)
        y64 = norm_rows(q_in, f32(w[0]), offset, eps, np.float64)
        top = np.abs(y64).max(-1, keepdims=True)
        y64 = turn(y64, rows, r, inter, np.float64)
        bound = np.abs(y64) * (torch.finfo(dt).eps / 2) * (1 + 2.0 ** -7) + 16 * U * 2 * top + torch.finfo(dt).tiny
        ok = np.abs(f32(qo) - y64) <= bound
        ok[list(skip)] = True
        assert ok.all()
    return qo, kc, vc


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,r,h", [(64, 64, 64), (64, 16, 16), (64, 48, 32), (128, 128, 128), (128, 64, 64),
                                   (128, 112, 128), (256, 256, 256), (256, 64, 32), (256, 208, 128)])
@pytest.mark.parametrize("T", [37, 3300])
def test_head_dims_and_parts(T, D, r, h, inter):
    """Few rows (a warp each) and many (the bulk form, whose lanes hold other elements)."""
    case = make(D + r, T, 6, 2, D, 16, r, BF)
    check(*case, 16, True, True, h, inter, False, w=gains(D, BF, 0.0))


@pytest.mark.parametrize("T,hq,hkv,P", [(1, 32, 8, 16), (2, 1, 1, 64), (255, 15, 3, 32), (600, 8, 8, 16),
                                        (1100, 32, 8, 64), (9001, 2, 1, 16)])
@pytest.mark.parametrize("dt,meta,wdt,offset,eps", [(BF, False, BF, 0.0, 1e-6), (F16, True, torch.float32, 1.0, 1e-5),
                                                    (BF, True, torch.float32, 0.0, 1e-2), (F16, False, F16, 1.0, 1e-6)])
def test_sizes_formats_and_gains(T, hq, hkv, P, dt, meta, wdt, offset, eps):
    case = make(T, T, hq, hkv, 128, P, 128, dt)
    check(*case, P, True, T % 2 == 0, 128, T % 3 == 0, meta, w=gains(128, wdt, offset), offset=offset, eps=eps)


@pytest.mark.parametrize("D,hq,hkv", [(64, 40, 5), (64, 65, 1), (128, 33, 3), (128, 64, 8), (256, 40, 2)])
def test_many_heads(D, hq, hkv):
    """More q-heads than an item takes, and a rest."""
    for T in (3, 700):
        case = make(D + hq, T, hq, hkv, D, 32, D, BF)
        check(*case, 32, True, True, 64, False, False, w=gains(D, torch.float32, 1.0), offset=1.0)


@pytest.mark.parametrize("T", [50, 3000])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_without_gains_q_or_v_and_in_place(D, T):
    q, k, v, pages, slots, pos, cs = make(3, T, 4, 2, D, 16, D // 2, BF)
    w, tail = gains(D, BF, 0.0), (16, True, True, 64, False, False)
    rest = (pages, slots, pos, cs)
    check(q, k, v, *rest, *tail, w=(None, None), offset=0.5)   # (an offset without gains is not used)
    check(q, k, v, *rest, *tail, w=(w[0], None))
    check(q, k, v, *rest, *tail, w=(None, w[1]))
    check(None, k, v, *rest, *tail, w=w)
    check(q, k, None, *rest, *tail, w=w)
    check(q, k, v, *rest, *tail, w=w, q_out=q)


@pytest.mark.parametrize("T", [64, 5000])
def test_padding_and_bad_entries(T):
    q, k, v, pages, slots, pos, cs = make(5, T, 8, 4, 128, 16, 128, BF)
    w = gains(128, BF, 0.0)
    slots[3] = slots[17] = slots[T - 1] = -1
    check(q, k, v, pages, slots, pos, cs, 16, True, True, 128, False, False, w=w)
    for at, val in ((slots, pages * 16), (slots, -2), (pos, cs.shape[0]), (pos, -1)):
        old = int(at[9])
        at[9] = val
        check(q, k, v, pages, slots, pos, cs, 16, True, True, 128, False, False, w=w,
              status=saw.SAW_ERR_DEVICE_INDEX, skip=[9] if at is pos else [])
        at[9] = old


@pytest.mark.parametrize("T", [40, 4000])
def test_extreme_rows(T):
    """Zero and constant rows, rows whose squares are below eps, and the largest ones."""
    q, k, v, pages, slots, pos, cs = make(6, T, 2, 2, 128, 16, 128, BF)
    for i, val in enumerate((0.0, -0.0, 1.0, -3.0e4, 1e-10, 6.0e4, 1e17)):
        k[i], q[i] = val, val
    k[7, :, 5], q[7, :, 5] = 5.0e4, -5.0e4
    for rk in (True, False):
        check(q, k, v, pages, slots, pos, cs, 16, rk, rk, 128, False, True, w=gains(128, torch.float32, 0.0))


def test_rows_of_either_form_are_the_same():
    """A row's bytes do not depend on how many rows the call has."""
    q, k, v, pages, slots, pos, cs = make(11, 4000, 8, 2, 128, 16, 96, BF)
    w = gains(128, BF, 0.0)
    a = run(q, k, v, *w, pages, slots, pos, cs, 16, True, True, 128)
    kc, vc = new_caches(pages, 16, 2, 128)
    qo = torch.empty_like(q)
    for i in range(0, 4000, 400):
        t = slice(i, i + 400)
        saw.saw_norm_rope_append(q[t], k[t], v[t], *w, pos[t], cs, slots[t], qo[t], kc, vc, pages, 16, True, True, 128)
    assert torch.equal(a[0], qo) and torch.equal(a[1], kc) and torch.equal(a[2], vc)


@pytest.mark.parametrize("T", [64, 5000])
def test_other_stream_and_graph(T):
    q, k, v, pages, slots, pos, cs = make(4, T, 8, 2, 128, 16, 128, BF)
    w = gains(128, BF, 0.0)
    args = (pages, slots, pos, cs, 16, True, True, 128)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a = run(q, k, v, *w, *args)
    b = run(q, k, v, *w, *args, stream=side)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))
    kc, vc = new_caches(pages, 16, 2, 128)
    qo = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_norm_rope_append(q, k, v, *w, pos, cs, slots, qo, kc, vc, pages, 16, True, True, 128)
    pos.copy_(pos.flip(0))
    w.mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    want = run(q, k, v, *w, *args)
    assert torch.equal(qo, want[0]) and torch.equal(kc, want[1]) and torch.equal(vc, want[2])


def test_no_tokens():
    q, k, v, pages, slots, pos, cs = make(4, 1, 8, 2, 128, 16, 128, BF)
    e = slice(0, 0)
    _, kc, _, st = run(q[e], k[e], v[e], None, None, pages, slots[e], pos[e], cs, 16, True, True, 128)
    assert st == 0 and (kc == 0xAB).all()
