"""saw_sparse_decode_int4 against 64 bits, over lists that differ per kv-head.

The bound, with v the largest 2-norm of a value row.  A base-2 logit is
1.44 sm_scale (s sum(n q') + z sum(q')): up to 17 binary32 sums and a few more
roundings, on partial sums of half of 15 s sum|q'| < 2^10.6 (unit-variance rows,
D <= 256, s <= 0.5).  Roundings of either sign leave about sqrt(20) 2^-24 2^9.6
1.44 / 16 = 2^-15.7 in the exponent (relative 2^-16.2 in a weight; smaller D
have smaller sums and a larger sm_scale, which is worse by at most 2), and an
output moves by at most twice a weight's change times v: 2^-14 v holds.  p s,
held to 22 bits, adds less than 2^-21 v.  A bfloat16 output takes p s in 11
bits: five standard deviations of that rounding (sparse_oracle.attend), and half
a step of the output's type.
"""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from sparse_oracle import attend

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def make(seed, lens, hq, hkv, D, P, dt, meta, rot_k=True, rot_v=True, h=64, spare=5):
    """lens [B][hkv]: tokens per list; every list its own pages, in any order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    B, width = lens.shape[0], max(int(-(-lens.max() // P)), 1) if lens.size else 1
    pages = max(width + spare, 8)
    tables = np.full((B, hkv, width), -1, np.int32)
    for b in range(B):
        for k in range(hkv):
            n = -(-int(lens[b, k]) // P)
            tables[b, k, :n] = rng.permutation(pages)[:n]
    T = pages * P
    k, v = (torch.randn(T, hkv, D, generator=g, device="cuda").to(dt) for _ in range(2))
    n = saw.saw_cache_bytes(pages, P, hkv, D)
    kc, vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    saw.saw_quantize_append(k, v, torch.arange(T, device="cuda").int(), kc, vc, pages, P, rot_k, rot_v, h, meta_bf16=meta)
    q = torch.randn(B, hq, D, generator=g, device="cuda").to(dt)
    return q, kc, vc, tables, lens, pages


def run(q, kc, vc, tables, lens, pages, P, rot_k, rot_v, h, meta, odt=None, max_len=None, ws=None, scale=0.0, stream=None):
    B, hq, D = q.shape
    hkv = tables.shape[1]
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    max_len = int(lens.max()) if max_len is None else max_len
    out = torch.full((B, hq, D), float("nan"), dtype=odt or q.dtype, device="cuda")
    if ws is None:
        need = saw.saw_sparse_decode_workspace_bytes(B, hq, hkv, D, P, max_len)
        ws = torch.zeros(need, dtype=torch.uint8, device="cuda") if need else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, kc, vc, i32(tables), i32(lens))
    torch.cuda.synchronize()
    saw.saw_sparse_decode_int4(*args, max_len, hkv, pages, P, rot_k, rot_v, h, out, ws, sm_scale=scale, dev_status=st,
                               stream=stream, meta_bf16=meta)
    torch.cuda.synchronize()
    return out, int(st.item())


def check(q, kc, vc, tables, lens, pages, P, rot_k, rot_v, h, meta, status=0, ref_lens=None, **kw):
    out, st = run(q, kc, vc, tables, lens, pages, P, rot_k, rot_v, h, meta, **kw)
    assert st == status
    D, hkv = q.shape[2], tables.shape[1]
    scale = kw.get("scale") or D ** -0.5
    ref, top, sd = attend(q.float().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), tables,
                          lens if ref_lens is None else ref_lens, hkv, D, P, rot_k, rot_v, h, scale, meta, pages)
    bound = 2.0 ** -14 * top + np.zeros_like(ref)
    if out.dtype != F32:
        bound += np.abs(ref) * (torch.finfo(out.dtype).eps / 2) * (1 + 2.0 ** -7) + torch.finfo(out.dtype).tiny
    if out.dtype == BF:
        bound += 5 * sd[..., None]
    err = np.abs(out.double().cpu().numpy() - ref)
    assert (err <= bound).all(), float((err / bound).max())
    return out


@pytest.mark.parametrize("odt", [None, F32])
@pytest.mark.parametrize("dt,meta", [(BF, False), (F16, True)])
@pytest.mark.parametrize("D,hq,hkv,P,h", [(64, 3, 3, 16, 64), (64, 12, 3, 64, 16), (64, 16, 2, 32, 32), (128, 8, 2, 16, 128),
                                          (128, 5, 1, 32, 16), (128, 24, 3, 64, 128), (256, 4, 2, 16, 256),
                                          (256, 14, 2, 64, 64)])
def test_formats_and_groups(D, hq, hkv, P, h, dt, meta, odt):
    rng = np.random.default_rng(D + hq)
    lens = rng.integers(1, 700, (5, hkv))
    lens[0, 0], lens[1] = 0, 1
    check(*make(D + hq + P, lens, hq, hkv, D, P, dt, meta, h=h), P, True, True, h, meta, odt=odt)


@pytest.mark.parametrize("rot_k,rot_v", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rotations_and_scale(D, rot_k, rot_v):
    case = make(D, [[77, 300], [0, 16]], 6, 2, D, 16, F16, False, rot_k, rot_v)
    check(*case, 16, rot_k, rot_v, 64, False)
    check(*case, 16, rot_k, rot_v, 64, False, scale=0.02)


@pytest.mark.parametrize("hq,D", [(2, 128), (8, 128), (16, 128), (8, 64), (4, 256)])
@pytest.mark.parametrize("B,n", [(1, 5000), (2, 1), (2, 15), (2, 17), (2, 16 * 40), (3, 2049), (180, 150), (400, 20),
                                 (190, 700)])
def test_lengths_and_grids(B, n, hq, D):
    """One token to several splits; grids of one wave, of 8-warp and of 4-warp CTAs."""
    rng = np.random.default_rng(n)
    lens = rng.integers(max(1, n - 40), n + 1, (B, 2))
    lens[0] = n
    check(*make(n + B, lens, hq, 2, D, 16, F16 if hq != 8 else BF, False), 16, True, True, 64, False)


def test_empty_lists():
    """No pages: a zero row; among others, alone, and a bound of zero tokens."""
    case = make(3, [[0, 50], [0, 0], [3000, 0]], 8, 2, 128, 16, BF, False)
    out = check(*case, 16, True, True, 64, False)
    assert (out[1] == 0).all() and (out[0, :4] == 0).all() and (out[2, 4:] == 0).all()
    case = make(3, [[0, 0]], 8, 2, 128, 16, F16, False)
    assert (check(*case, 16, True, True, 64, False) == 0).all()
    assert (check(*case, 16, True, True, 64, False, max_len=16, odt=F32) == 0).all()


def test_a_page_twice_counts_twice():
    q, kc, vc, tables, lens, pages = make(8, [[64, 48]], 4, 2, 128, 16, F16, False)
    tables[0, 0, 2] = tables[0, 0, 0]
    check(q, kc, vc, tables, lens, pages, 16, True, True, 64, False)


def test_bad_entries_are_skipped_and_reported():
    q, kc, vc, tables, lens, pages = make(9, [[640, 100], [300, 333], [2000, 16]], 8, 2, 128, 16, F16, False)
    bad = saw.SAW_ERR_DEVICE_INDEX
    t = tables.copy()
    t[0, 0, 7], t[2, 0, 100], t[1, 1, 20] = -1, pages, 2 ** 31 - 1
    check(q, kc, vc, t, lens, pages, 16, True, True, 64, False, status=bad)
    for v in (-1, 2001):
        L, R = lens.copy(), lens.copy()
        L[1, 1], R[1, 1] = v, 0
        check(q, kc, vc, tables, L, pages, 16, True, True, 64, False, status=bad, ref_lens=R, max_len=2000)


def test_whole_sequences_are_the_plain_decode():
    """Every page of a sequence for every kv-head: saw_paged_decode_int4's float32 output but for the
    rounding of p s, which the lists' form carries to 22 bits."""
    rng = np.random.default_rng(1)
    lens = np.repeat(rng.integers(1, 1500, (6, 1)), 2, 1).astype(np.int32)
    q, kc, vc, tables, _, pages = make(2, lens, 8, 2, 128, 16, BF, False)
    tables[:, 1] = tables[:, 0]
    got = check(q, kc, vc, tables, lens, pages, 16, True, True, 64, False, odt=F32)
    bt = torch.from_numpy(tables[:, 0].copy()).cuda()
    out = torch.empty_like(got)
    n = saw.saw_decode_workspace_bytes(6, 8, 2, 128, 16, int(lens.max()))
    ws = torch.zeros(max(n, 16), dtype=torch.uint8, device="cuda")
    saw.saw_paged_decode_int4(q, kc, vc, bt, torch.from_numpy(lens[:, 0].copy()).cuda(), int(lens.max()), 2, pages, 16, True,
                              True, 64, out, ws)
    _, _, sd = attend(q.float().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy(), tables, lens, 2, 128, 16, True, True, 64,
                      128 ** -0.5, False, pages)
    assert (np.abs((got - out).cpu().numpy()) <= 5 * sd[..., None] + 1e-3).all()


def test_one_workspace_for_calls_of_other_sizes():
    """A workspace serves the next call, whatever its sizes; the same call gives the same bytes."""
    big = make(4, [[5000] * 2] * 2, 16, 2, 128, 16, F16, False)
    small = make(5, [[3000, 1700]], 8, 2, 64, 16, F16, False)
    need = max(saw.saw_sparse_decode_workspace_bytes(2, 16, 2, 128, 16, 5000),
               saw.saw_sparse_decode_workspace_bytes(1, 8, 2, 64, 16, 3000))
    assert saw.saw_sparse_decode_workspace_bytes(1, 8, 2, 64, 16, 3000) > 0
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    a = [check(*c, 16, True, True, 64, False, ws=ws) for c in (big, small, big, small)]
    assert torch.equal(a[0], a[2]) and torch.equal(a[1], a[3])


def test_other_stream_and_graph():
    q, kc, vc, tables, lens, pages = make(6, [[3000, 1700], [40, 0]], 8, 2, 128, 16, BF, False)
    want = check(q, kc, vc, tables, lens, pages, 16, True, True, 64, False)
    got, _ = run(q, kc, vc, tables, lens, pages, 16, True, True, 64, False, stream=torch.cuda.Stream())
    assert torch.equal(got, want)
    need = saw.saw_sparse_decode_workspace_bytes(2, 8, 2, 128, 16, 3000)
    ws, out = torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    t, ln = torch.from_numpy(tables).cuda(), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_sparse_decode_int4(q, kc, vc, t, ln, 3000, 2, pages, 16, True, True, 64, out, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert (out == 0).all()
    ln.copy_(torch.from_numpy(lens))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
