"""saw_select_pages against the rule in whole numbers: the lists are equal, entry
by entry, at every format and size, with ties, odd scores and bad entries."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from sparse_oracle import quantize, select, summary_rows, summary_stride

pytestmark = pytest.mark.gpu
BF, F16 = torch.bfloat16, torch.float16


def make(seed, lens, hq, hkv, D, P, dt, meta, spare=3, spread=0.4):
    rng = np.random.default_rng(seed)
    need = [-(-int(L) // P) for L in lens]
    pages = sum(need) + spare
    bt, at, order = np.full((len(lens), max(need + [1])), -1, np.int32), 0, rng.permutation(pages)
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    x = (spread * rng.standard_normal((pages, hkv, D)) + rng.standard_normal((hkv, D))).astype(np.float32)
    s = np.zeros(pages * summary_stride(hkv, D), np.uint8)
    codes, words = summary_rows(s, hkv, D)
    c, w = quantize(x, meta)
    row = s.reshape(pages, -1)
    row[:, :hkv * D // 2] = c.reshape(pages, -1)
    row[:, hkv * D // 2:hkv * (D // 2 + 4)] = w.reshape(pages, -1)
    q = torch.from_numpy(rng.standard_normal((len(lens), hq, D)).astype(np.float32) * 2).to(dt).cuda()
    return q, s, bt, pages


def run(q, s, bt, lens, hkv, P, pages, rotate, h, take, first, last, meta, max_len=None, stream=None):
    B = len(lens)
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    full = lambda *n: torch.full(n, -7, dtype=torch.int32, device="cuda")
    tables, page_nos, out, st = full(B, hkv, take), full(B, hkv, take), full(B, hkv), torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (q, torch.from_numpy(s).cuda(), i32(bt), i32(lens), int(max(lens, default=0)) if max_len is None else max_len)
    torch.cuda.synchronize()
    saw.saw_select_pages(*args, hkv, pages, P, rotate, h, first, last, tables, out, sel_pages=page_nos, dev_status=st,
                         stream=stream, meta_bf16=meta)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (tables, page_nos, out)], int(st.item())


def check(q, s, bt, pages, lens, hkv, P, rotate, h, take, first, last, meta, status=0, as_lens=None, **kw):
    got, st = run(q, s, bt, lens, hkv, P, pages, rotate, h, take, first, last, meta, **kw)
    assert st == status
    want = select(q.float().cpu().numpy(), s, bt, lens if as_lens is None else as_lens, hkv, q.shape[2], P, rotate, h,
                  take, first, last, meta)
    for g, w, what in zip(got, want, ("tables", "pages", "lens")):
        assert np.array_equal(g, w), what
    return got


@pytest.mark.parametrize("dt,meta", [(BF, False), (F16, True)])
@pytest.mark.parametrize("D,h", [(64, 64), (64, 16), (128, 128), (128, 0), (256, 256), (256, 32)])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 3), (15, 3), (16, 2)])
def test_formats_and_groups(D, h, hq, hkv, dt, meta):
    lens = [1, 16, 17, 500, 1023, 1024, 40 * 16]
    case = make(D + h + hq, lens, hq, hkv, D, 16, dt, meta)
    check(*case, lens, hkv, 16, h > 0, h or 16, 20, 1, 2, meta)


@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("take,first,last", [(1, 0, 1), (2, 0, 1), (2, 1, 1), (9, 4, 4), (33, 0, 16), (64, 1, 1),
                                             (65, 3, 5), (300, 1, 2)])
def test_counts(P, take, first, last):
    """Lists without a scored page, one scored page, more than a sequence has; lengths at their borders."""
    lens = [0, 1, P, take * P - 1, take * P, take * P + 1, (take + 1) * P, (take + 2) * P + 5, 70 * P - 3]
    case = make(P + take, lens, 8, 2, 128, P, BF, False)
    check(*case, lens, 2, P, True, 128, take, first, last, False)


@pytest.mark.parametrize("B,L,take", [(1, 20000, 128), (1, 70000, 500), (3, 40000, 17), (40, 6000, 64), (160, 2100, 40),
                                      (1, 4 * 16 * 4096, 2000)])
def test_long_and_many(B, L, take):
    """One cluster and one CTA per list; runs of pages that end inside a tile."""
    rng = np.random.default_rng(B)
    lens = [L] + [int(x) for x in rng.integers(1, L, B - 1)]
    case = make(B + L, lens, 4, 2, 64, 16, BF, False)
    check(*case, lens, 2, 16, True, 64, take, 1, 3, False)


@pytest.mark.parametrize("hkv", [4, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("D,B,L", [(64, 1, 9000), (128, 3, 5000), (256, 1, 3000), (128, 90, 700), (128, 200, 500), (64, 40, 2500)])
def test_kv_heads(D, B, L, hkv):
    """Many kv-heads to a sequence: clusters and single CTAs that share its rows, and sizes beyond them."""
    if B > 3 and hkv > 9:
        B = 20
    rng = np.random.default_rng(hkv)
    lens = [L] + [int(x) for x in rng.integers(1, L, B - 1)]
    case = make(B + L, lens, 2 * hkv, hkv, D, 16, BF, hkv % 2 == 1)
    check(*case, lens, hkv, 16, True, 64, 21, 1, 2, hkv % 2 == 1)


@pytest.mark.parametrize("hkv", [1, 8])
def test_longest(hkv):
    """As many pages as a call takes."""
    lens = [16 * (1 << 18), 16 * 200000 + 5]
    q, s, bt, pages = make(1, [40000, 30000], hkv, hkv, 64, 16, BF, False)
    t = np.stack([np.resize(bt[0, :2500], 1 << 18), np.resize(bt[1, :1875], 1 << 18)]).astype(np.int32)
    check(q, s, t, pages, lens, hkv, 16, True, 64, 300, 1, 2, False)


@pytest.mark.parametrize("L", [4000, 40000])
def test_ties_go_to_the_lower_page(L):
    """Few different summaries, so that most scores are equal; all equal; all zero (and -0 beside 0)."""
    lens = [L, L - 37]
    q, s, bt, pages = make(3, lens, 8, 2, 128, 16, BF, False)
    row = s.reshape(pages, -1)
    for kinds in (3, 1):
        row[:] = row[np.arange(pages) % kinds]
        for take in (5, 100):
            check(q, s, bt, pages, lens, 2, 16, True, 128, take, 1, 2, False)
    check(torch.zeros_like(q), s, bt, pages, lens, 2, 16, True, 128, 60, 1, 2, False)
    codes, words = summary_rows(s, 2, 128)
    row[:, :2 * 64] = 0                                  # codes 0: score qs z J
    w = row[:, 128:136].reshape(pages, 2, 4)
    w[:, :, 2:] = np.array([0x00, 0x80], np.uint8)       # z = -0
    w[::2, :, 2:] = 0
    row[:, 128:136] = w.reshape(pages, 8)
    check(q, s, bt, pages, lens, 2, 16, True, 128, 60, 1, 2, False)


def test_scores_that_are_no_numbers():
    """Infinite and NaN words, infinite and NaN queries, scores that overflow: -infinity for a NaN."""
    lens = [3000, 2000, 1500, 900]
    q, s, bt, pages = make(9, lens, 8, 2, 128, 16, BF, True)
    row = s.reshape(pages, -1)
    w = row[:, 128:136].copy().view(np.uint16).reshape(pages, 2, 2)
    for i, bad in enumerate((0x7F80, 0xFF80, 0x7FC0, 0x7F00, 0xFF00)):
        w[i::11, :, i & 1] = bad
    row[:, 128:136] = w.view(np.uint8).reshape(pages, 8)
    q[1, 2, 7] = float("nan")
    q[2, 1, 3] = float("inf")
    q[2, 5:7] = 3e38
    q[3, 0:4] = 1e-42
    with np.errstate(all="ignore"):
        for rotate in (True, False):
            check(q, s, bt, pages, lens, 2, 16, rotate, 128, 30, 1, 2, True)


def test_bad_entries():
    """A length out of range gives an empty list; a bad page id scores last; both are reported."""
    lens = [700, 640, 333]
    q, s, bt, pages = make(5, lens, 4, 2, 128, 16, BF, False)
    bad = saw.SAW_ERR_DEVICE_INDEX
    check(q, s, bt, pages, [700, -1, 333], 2, 16, True, 128, 12, 1, 2, False, status=bad, as_lens=[700, 0, 333], max_len=704)
    check(q, s, bt, pages, [700, 640, 333], 2, 16, True, 128, 12, 1, 2, False, status=bad, as_lens=[0, 640, 333],
          max_len=699)
    t = bt.copy()
    t[0, 5], t[0, 9], t[1, 20] = -1, pages, 2 ** 31 - 1
    check(q, s, t, pages, lens, 2, 16, True, 128, 12, 1, 2, False, status=bad)
    check(q, s, t, pages, lens, 2, 16, True, 128, 42, 1, 2, False, status=bad)


def test_all_rows_short_and_without_page_numbers():
    lens = [100, 0, 33]
    q, s, bt, pages = make(5, lens, 4, 2, 128, 16, BF, False)
    got = check(q, s, bt, pages, lens, 2, 16, True, 128, 12, 1, 2, False)
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    tables, out = torch.zeros(3, 2, 12, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    saw.saw_select_pages(q, torch.from_numpy(s).cuda(), i32(bt), i32(lens), 112, 2, pages, 16, True, 128, 1, 2, tables, out)
    assert np.array_equal(tables.cpu().numpy(), got[0]) and np.array_equal(out.cpu().numpy(), got[2])


def test_other_stream_and_graph():
    lens = [3000, 2500, 100]
    q, s, bt, pages = make(5, lens, 8, 2, 128, 16, BF, False)
    want = check(q, s, bt, pages, lens, 2, 16, True, 128, 12, 1, 2, False)
    got, _ = run(q, s, bt, lens, 2, 16, pages, True, 128, 12, 1, 2, False, stream=torch.cuda.Stream())
    assert all(np.array_equal(a, b) for a, b in zip(got, want))
    z = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    tables, out, ln, t, sd = z(3, 2, 12), z(3, 2), z(3), torch.from_numpy(bt).cuda(), torch.from_numpy(s).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_select_pages(q, sd, t, ln, 3000, 2, pages, 16, True, 128, 1, 2, tables, out)
    ln.copy_(torch.tensor(lens))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(tables.cpu().numpy(), want[0]) and np.array_equal(out.cpu().numpy(), want[2])


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,hkv,L", [(13, 8, 20000), (30, 8, 9000), (60, 8, 8500), (80, 8, 4000), (8, 8, 20000)])
def test_cta_shapes(B, hkv, L, D, ties):
    """Grids that take 16-warp CTAs, 8-warp ones with either register count, 4-warp ones and
    clusters; few different summaries, so that a histogram cannot part them, or many."""
    rng = np.random.default_rng(B + D)
    lens = [L] + [int(x) for x in rng.integers(L // 2, L, B - 1)]
    q, s, bt, pages = make(B + D, lens[:3], hkv, hkv, D, 16, BF, False)
    # (the sequences share the first three's pages)
    t = np.full((B, bt.shape[1]), -1, np.int32)
    for b in range(B):
        t[b, :-(-lens[b] // 16)] = rng.permutation(pages)[:-(-lens[b] // 16)]
    q = torch.from_numpy(rng.standard_normal((B, hkv, D)).astype(np.float32)).to(BF).cuda()
    if ties:
        row = s.reshape(pages, -1)
        row[:] = row[np.arange(pages) % 2]
    check(q, s, t, pages, lens, hkv, 16, True, 64, 70, 1, 2, False)
