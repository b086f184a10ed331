"""saw_build_tables against the definition, request by request in Python:
every word equal."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw

pytestmark = pytest.mark.gpu
KEEP = -7  # what the outputs hold before the call


def model(cached, new, free, nfree, P, pages, max_blocks, T, src, rows, bt):
    """The definition.  Returns the outputs and the set of codes that may be reported."""
    B = len(new)
    bt, status = bt.copy(), set()
    lens, cu = np.zeros(B, np.int32), np.zeros(B + 1, np.int32)
    slots, pos = np.full(T, -1, np.int32), np.zeros(T, np.int32)
    off = taken = t = 0
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        r = int(rows[b]) if rows is not None else b
        old = -(-c // P) if c >= 0 else 0
        ok = c >= 0 and n >= 0 and c + n <= max_blocks * P
        if ok and c > 0:
            ok = src is not None and 0 <= r < len(src) and old <= src.shape[1]
        tokens = max(n, 0)
        cu[b + 1] = cu[b] + tokens
        if not ok:
            status.add(saw.SAW_ERR_DEVICE_INDEX)
            t += tokens
            continue
        need = -(-(c + n) // P) - old
        fits = need == 0 or off + need <= nfree
        if old:
            bt[b, :old] = src[r, :old]
        lens[b] = c + n if fits else c
        if not fits:
            status.add(saw.SAW_ERR_DEVICE_PAGES)
        entry = {}
        for e in range(need if fits else 0):
            v = int(free[off + e])
            if not 0 <= v < pages:
                v = -1
                status.add(saw.SAW_ERR_DEVICE_INDEX)
            bt[b, old + e] = v
            entry[old + e] = v
            taken = off + e + 1
        for i in range(tokens):
            if fits and t < T:
                lp = (c + i) // P
                v = entry.get(lp, int(src[r, lp]) if lp < old else -1)
                pos[t] = c + i
                if 0 <= v < pages:
                    slots[t] = v * P + (c + i) % P
                else:
                    status.add(saw.SAW_ERR_DEVICE_INDEX)
            t += 1
        off += need
    if t > T:
        status.add(saw.SAW_ERR_DEVICE_INDEX)
    return dict(bt=bt, lens=lens, cu=cu, slots=slots, pos=pos, taken=np.array([taken], np.int32)), status


def run(cached, new, free, nfree, P, pages, max_blocks, T, src=None, rows=None, bt=None, in_place=False,
        stream=None):
    dev = "cuda"
    g = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)
    B = len(new)
    s = g(src)
    out = dict(bt=s if in_place else g(bt), lens=torch.full((B,), KEEP, dtype=torch.int32, device=dev),
               cu=torch.full((B + 1,), KEEP, dtype=torch.int32, device=dev),
               slots=torch.full((T,), KEEP, dtype=torch.int32, device=dev),
               pos=torch.full((T,), KEEP, dtype=torch.int32, device=dev),
               taken=torch.full((1,), KEEP, dtype=torch.int32, device=dev))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    torch.cuda.synchronize()
    saw.saw_build_tables(g(cached), g(new), g(free), None if nfree is None else g([nfree]), P, pages,
                         out["bt"], out["lens"], out["cu"], out["slots"], out["pos"], out["taken"],
                         src_tables=s, src_rows=g(rows), dev_status=status, stream=stream)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}, int(status.item())


def check(cached, new, free, nfree, P, pages, max_blocks, T, src=None, rows=None, in_place=False):
    B = len(new)
    bt = src[:B] if in_place else np.full((B, max_blocks), KEEP, np.int32)
    c = np.zeros(B, np.int64) if cached is None else cached
    want, codes = model(c, new, free, len(free) if nfree is None else nfree, P, pages, max_blocks, T, src, rows, bt)
    got, status = run(cached, new, free, nfree, P, pages, max_blocks, T, src, rows, bt, in_place)
    for k in want:
        w = want[k]
        assert np.array_equal(got[k][:len(w)], w), (k, np.argwhere(got[k][:len(w)] != w)[:5])
        assert np.array_equal(got[k][len(w):], src[len(w):] if k == "bt" and in_place else got[k][len(w):])
    assert status in codes if codes else status == 0
    return got, status


def batch(seed, B, hi, new, P, spare=3, extra_rows=2):
    rng = np.random.default_rng(seed)
    cached, fresh = rng.integers(0, hi + 1, B), rng.integers(0, new + 1, B)
    old = -(-cached // P)
    need = -(-(cached + fresh) // P) - old
    pages = int(old.sum() + need.sum()) + spare
    ids = rng.permutation(pages).astype(np.int32)
    blocks = int((old + need).max()) + 2 if B else 2
    src = np.full((B + extra_rows, blocks), -1, np.int32)
    rows = rng.permutation(B + extra_rows)[:B]
    at = 0
    for b in range(B):
        src[rows[b], :old[b]] = ids[at:at + old[b]]
        at += old[b]
    return cached, fresh, ids[at:], pages, blocks, src, rows


@pytest.mark.parametrize("B,hi,new,P", [
    (1, 0, 1, 16), (1, 5000, 700, 16), (3, 40, 40, 32), (31, 100, 3, 64), (32, 100, 1, 16), (33, 100, 1, 16),
    (64, 3000, 1, 16), (511, 200, 9, 32), (513, 300, 5, 16), (4096, 60, 2, 16), (4097, 60, 2, 16),
    (20001, 40, 2, 16),
])
def test_gathered(B, hi, new, P):
    cached, fresh, free, pages, blocks, src, rows = batch(B + P, B, hi, new, P)
    check(cached, fresh, free, None, P, pages, blocks, int(fresh.sum()) + 5, src, rows)


@pytest.mark.parametrize("B,hi,new,P", [(5, 100, 33, 16), (70, 900, 2, 32), (4500, 30, 2, 16)])
def test_in_place(B, hi, new, P):
    cached, fresh, free, pages, blocks, src, rows = batch(B, B, hi, new, P, extra_rows=0)
    src = np.ascontiguousarray(src[rows])
    check(cached, fresh, free, len(free), P, pages, blocks, int(fresh.sum()), src, None, in_place=True)


def test_fresh_batch_without_tables():
    """Nothing cached: no source tables, no cached lengths; a prompt of many pages."""
    new = np.array([1, 0, 70001, 16, 17])
    pages = int((-(-new // 16)).sum())
    check(None, new, np.random.default_rng(0).permutation(pages), None, 16, pages, 4400, int(new.sum()) + 30)


@pytest.mark.parametrize("B", [40, 5000])
def test_free_list_runs_out(B):
    cached, fresh, free, pages, blocks, src, rows = batch(3, B, 50, 40, 16)
    for nfree in (0, 1, len(free) // 2, len(free) - 4):
        got, status = check(cached, fresh, free, nfree, 16, pages, blocks, int(fresh.sum()), src, rows)
        assert status == saw.SAW_ERR_DEVICE_PAGES
        assert got["taken"][0] <= nfree


def test_forked_rows_share_their_pages():
    """Three requests continue one row whose pages are full: the same pages first, their own after."""
    src = np.array([[4, 2, 9, -1], [7, -1, -1, -1]], np.int32)
    got, _ = check([32, 32, 32, 3], [1, 17, 16, 1], [11, 12, 13, 14, 15, 16], None, 16, 20, 4, 40, src,
                   [0, 0, 0, 1])
    assert got["bt"][0, :3].tolist() == [4, 2, 11] and got["bt"][1, :4].tolist() == [4, 2, 12, 13]


@pytest.mark.parametrize("what", ["neg_cached", "neg_new", "too_long", "row", "row_neg", "src_blocks", "free_id",
                                  "src_id", "tokens", "count"])
def test_bad_input_is_reported_and_skipped(what):
    cached, fresh, free, pages, blocks, src, rows = batch(11, 37, 200, 20, 16)
    cached[3], fresh[3], cached[8] = 30, 5, 17
    free, nfree, T = np.array(free), None, int(np.maximum(fresh, 0).sum())
    if what == "neg_cached":
        cached[3] = -1
    elif what == "neg_new":
        fresh[3] = -2
    elif what == "too_long":
        fresh[3] = blocks * 16
    elif what == "row":
        rows[3] = len(src)
    elif what == "row_neg":
        rows[3] = -1
    elif what == "src_blocks":
        blocks, cached[3] = blocks + 9, blocks * 16 + 1
    elif what == "free_id":
        free[1], free[2] = pages, -1
    elif what == "src_id":
        src[rows[8], 1] = -1
        fresh[8] = 4
    elif what == "tokens":
        T -= 9
    elif what == "count":
        nfree = len(free) + 1
    if what == "count":  # more than the list holds: reported, the list's length counts
        want, _ = model(cached, fresh, free, len(free), 16, pages, blocks, T, src, rows,
                        np.full((37, blocks), KEEP, np.int32))
        got, status = run(cached, fresh, free, nfree, 16, pages, blocks, T, src, rows,
                          np.full((37, blocks), KEEP, np.int32))
        assert all(np.array_equal(got[k], want[k]) for k in want)
    else:
        _, status = check(cached, fresh, free, nfree, 16, pages, blocks, T, src, rows)
    assert status in (saw.SAW_ERR_DEVICE_INDEX, saw.SAW_ERR_DEVICE_PAGES)


def test_lengths_that_overflow():
    """Sums beyond 2^31 tokens: refused requests keep their counts, and nothing is written out of range."""
    new = np.array([2**31 - 1, 2**31 - 1, 5, 2**31 - 1])
    got, status = run(None, new, np.arange(4), None, 16, 4, 3, 20, bt=np.full((4, 3), KEEP, np.int32))
    assert status == saw.SAW_ERR_DEVICE_INDEX
    assert got["lens"].tolist() == [0, 0, 5, 0]
    assert got["cu"].tolist() == [0] + [2**31 - 1] * 4
    assert (got["slots"] == -1).all() and got["taken"][0] == 1 and got["bt"][2, 0] == 0


def test_empty_batch_pads():
    t = lambda *s: torch.full(s, KEEP, dtype=torch.int32, device="cuda")
    cu, slots, pos, taken = t(1), t(70), t(70), t(1)
    saw.saw_build_tables(None, t(0), t(4), None, 16, 8, t(0, 3), t(0), cu, slots, pos, taken)
    assert cu.item() == 0 and taken.item() == 0 and (slots == -1).all() and (pos == 0).all()


def test_other_stream_and_graph_replay():
    """A captured call reads its lengths at replay; one on another stream gives the same."""
    cached, fresh, free, pages, blocks, src, rows = batch(5, 50, 300, 4, 16)
    T = 50 * 4
    bt = np.full((50, blocks), KEEP, np.int32)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got, status = run(cached, fresh, free, None, 16, pages, blocks, T, src, rows, bt)
    want, _ = model(cached, fresh, free, len(free), 16, pages, blocks, T, src, rows, bt)
    assert status == 0 and all(np.array_equal(got[k], want[k]) for k in want)
    g = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    d = dict(c=g(cached), n=g(fresh), f=g(free), bt=g(bt), s=g(src), r=g(rows))
    o = [torch.zeros(k, dtype=torch.int32, device="cuda") for k in (50, 51, T, T, 1)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_build_tables(d["c"], d["n"], d["f"], None, 16, pages, d["bt"], *o, src_tables=d["s"], src_rows=d["r"])
    fresh2 = fresh[::-1].copy()
    cached2 = np.maximum(cached - 4, 0)
    d["n"].copy_(g(fresh2))
    d["c"].copy_(g(cached2))
    graph.replay()
    torch.cuda.synchronize()
    want, _ = model(cached2, fresh2, free, len(free), 16, pages, blocks, T, src, rows, bt)
    for k, v in zip(("lens", "cu", "slots", "pos", "taken"), o):
        assert np.array_equal(v.cpu().numpy(), want[k]), k
    assert np.array_equal(d["bt"].cpu().numpy(), want["bt"])
