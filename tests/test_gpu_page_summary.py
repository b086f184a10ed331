"""saw_page_summary against the rule step by step in binary32, byte for byte:
pages that a step completes and no others, every format and size, and the bytes
around a summary."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from gpu_helpers import SENTINEL, assert_bytes_equal
from sparse_oracle import page_mean, rows_of, summaries, summary_rows, word_value

pytestmark = pytest.mark.gpu


def filled(seed, pages, hkv, D, P, meta, dt=torch.bfloat16):
    """A K cache of whole pages with heavy-tailed rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = pages * P
    k = torch.randn(T, hkv, D, generator=g, device="cuda")
    k *= torch.rand(T, 1, 1, generator=g, device="cuda") * 3
    k[:, :, 5] *= 9
    kc = torch.empty(saw.saw_cache_bytes(pages, P, hkv, D), dtype=torch.uint8, device="cuda")
    saw.saw_quantize_append(k.to(dt), None, torch.arange(T, device="cuda").int(), kc, None, pages, P, True, False,
                            64, meta_bf16=meta)
    return kc


def tables(seed, lens, P, pages, width):
    order = np.random.default_rng(seed).permutation(pages)
    bt, at = np.full((len(lens), width), -1, np.int32), 0
    for b, L in enumerate(lens):
        n = -(-L // P)
        bt[b, :n] = order[at:at + n]
        at += n
    return bt


def run(kc, bt, lens, new, hkv, D, P, pages, meta, max_new=None, stream=None):
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")
    out = torch.full((saw.saw_summary_bytes(pages, hkv, D) + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    if max_new is None:
        max_new = max((min(n, L) for n, L in zip(lens if new is None else new, lens)), default=0)
    args = (kc, i32(bt), i32(lens), None if new is None else i32(new), max_new, hkv, D, pages, P, out)
    torch.cuda.synchronize()
    saw.saw_page_summary(*args, dev_status=st, meta_bf16=meta, stream=stream)
    torch.cuda.synchronize()
    return out, int(st.item())


def check(kc, bt, lens, new, hkv, D, P, pages, meta, **kw):
    out, st = run(kc, bt, lens, new, hkv, D, P, pages, meta, **kw)
    assert st == 0
    want = np.full(out.numel(), SENTINEL, np.uint8)
    summaries(want[:-64], kc.cpu().numpy(), bt, lens, new, hkv, D, P, meta)
    assert_bytes_equal(out, want, "summaries")
    return out


@pytest.mark.parametrize("meta", [False, True])
@pytest.mark.parametrize("P", [16, 32, 64])
@pytest.mark.parametrize("D,hkv", [(64, 1), (64, 3), (64, 8), (128, 1), (128, 5), (256, 2), (256, 3)])
def test_formats_and_sizes(D, hkv, P, meta):
    lens = [5 * P + 3, P, P - 1, 0, 2 * P, 3 * P + 1, 1]
    new = [5 * P + 3, 1, P - 1, 0, P + 1, 2, 1]
    pages = 16
    check(filled(D + hkv + P, pages, hkv, D, P, meta), tables(P, lens, P, pages, 8), lens, new, hkv, D, P, pages, meta)


@pytest.mark.parametrize("new", [1, 2, 15, 16, 17, 33, None])
def test_a_page_is_written_when_it_is_completed(new):
    """Every length around a page's end; whole prompts with None or with counts above the lengths."""
    P, hkv, D = 16, 2, 128
    lens = list(range(0, 2 * P + 3)) + [1000]
    pages = sum(-(-n // P) for n in lens) + 2
    kc, bt = filled(1, pages, hkv, D, P, False), tables(2, lens, P, pages, 64)
    n = None if new is None else [new] * len(lens)
    check(kc, bt, lens, n, hkv, D, P, pages, False)
    if new == 33:
        check(kc, bt, lens, [10 ** 9] * len(lens), hkv, D, P, pages, False)


def test_many_sequences_and_a_long_one():
    P, hkv, D = 16, 8, 128
    lens = [100] * 150 + [9000]
    pages = 7 * 150 + 563 + 1
    kc, bt = filled(4, pages, hkv, D, P, False), tables(5, lens, P, pages, 563)
    check(kc, bt, lens, [5] * 150 + [700], hkv, D, P, pages, False)


def test_the_mean():
    """The row is within half a step, and the roundings of the sums, of the mean in 64 bits."""
    P, hkv, D, pages = 32, 2, 128, 6
    kc = filled(3, pages, hkv, D, P, False)
    bt, lens = np.arange(pages, dtype=np.int32)[None], [pages * P]
    out, _ = run(kc, bt, lens, None, hkv, D, P, pages, False)
    codes, words = summary_rows(out.cpu().numpy()[:-64], hkv, D)
    for e in range(pages):
        for h in range(hkv):
            code, s, z = (x.astype(np.float64) for x in rows_of(kc.cpu().numpy(), e, h, hkv, D, P, False))
            mean = (code * s[:, None] + z[:, None]).mean(0)
            sc, zz = word_value(words[e, h].copy().view(np.uint16), False).astype(np.float64)
            got = np.empty(D)
            got[0::2], got[1::2] = codes[e, h] & 15, codes[e, h] >> 4
            # at most P + 3 roundings of a partial sum, each below the sum of magnitudes
            slack = (P + 3) * 2.0 ** -24 * ((code * s[:, None]).sum(0) + np.abs(z).sum()) / P
            assert (np.abs(got * sc + zz - mean) <= sc / 2 * (1 + 2.0 ** -10) + slack).all()
            assert np.abs(page_mean(kc.cpu().numpy(), e, h, hkv, D, P, False) - mean).max() <= slack.max()


def test_bad_entries_are_skipped_and_reported():
    P, hkv, D, pages = 16, 2, 128, 12
    kc = filled(6, pages, hkv, D, P, False)
    bt = np.arange(12, dtype=np.int32).reshape(3, 4)
    for lens, new, skip in (([64, -1, 20], [64, 1, 20], 1), ([64, 65, 20], [64, 1, 20], 1),
                            ([64, 40, 20], [64, -1, 20], 1), ([64, 40, 20], [20, 21, 20], 0)):
        out, st = run(kc, bt, lens, new, hkv, D, P, pages, False, max_new=64 if skip else 21 - 1)
        assert st == saw.SAW_ERR_DEVICE_INDEX
        good = list(lens)
        if skip:
            good[1] = 0
            new = [new[0], 0, new[2]]
        else:
            good[1] = 0
        want = np.full(out.numel(), SENTINEL, np.uint8)
        summaries(want[:-64], kc.cpu().numpy(), bt, good, [min(a, b) for a, b in zip(new, good)], hkv, D, P, False)
        assert_bytes_equal(out, want, f"{lens} {new}")
    for bad in (-1, pages):
        t = bt.copy()
        t[1, 1] = bad
        out, st = run(kc, t, [64, 40, 20], None, hkv, D, P, pages, False)
        assert st == saw.SAW_ERR_DEVICE_INDEX
        want = np.full(out.numel(), SENTINEL, np.uint8)
        summaries(want[:-64], kc.cpu().numpy(), t, [64, 16, 20], None, hkv, D, P, False)
        assert_bytes_equal(out, want, f"page {bad}")


def test_nothing_new_and_no_sequences():
    kc, bt = filled(6, 4, 2, 128, 16, False), np.arange(4, dtype=np.int32)[None]
    out, st = run(kc, bt, [64], [0], 2, 128, 16, 4, False, max_new=0)
    assert st == 0 and (out == SENTINEL).all()
    out, st = run(kc, bt[:0], [], [], 2, 128, 16, 4, False, max_new=64)
    assert st == 0 and (out == SENTINEL).all()


def test_other_stream_and_graph():
    P, hkv, D, pages = 16, 4, 128, 40
    kc, lens = filled(7, pages, hkv, D, P, False), [200, 100, 64]
    bt = tables(8, lens, P, pages, 16)
    want = check(kc, bt, lens, None, hkv, D, P, pages, False)
    out, _ = run(kc, bt, lens, None, hkv, D, P, pages, False, stream=torch.cuda.Stream())
    assert torch.equal(out, want)
    ln, t = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.from_numpy(bt).cuda()
    out = torch.full_like(want, SENTINEL)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        saw.saw_page_summary(kc, t, ln, None, 200, hkv, D, pages, P, out)
    ln.copy_(torch.tensor(lens))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
