"""saw_select_pages where no score is a finite number, and its lists against the
scores in 64 bits of the unrounded queries."""
import numpy as np
import pytest
import torch

from sparse_oracle import matrix, summary_rows, word_value
from test_gpu_select_pages import check, make, run

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("B,L", [(1, 20000), (30, 18000), (50, 9000), (90, 2500)])
@pytest.mark.parametrize("D", [64, 128])
def test_no_finite_score(B, L, D):
    """Every scored page of a list at -infinity (NaN queries, or words of infinity): the first pages in order;
    a cluster and CTAs of 16, 8 and 4 warps; and lists beside them whose scores are finite."""
    hkv = 4
    lens = [L - 16 * (b % 3) for b in range(B)]
    q, s, bt, pages = make(B + D, lens[:2], 2 * hkv, hkv, D, 16, BF, False)
    t = np.stack([np.resize(bt[b % 2, :-(-lens[b % 2] // 16)], bt.shape[1]) for b in range(B)]).astype(np.int32)
    q = torch.randn(B, 2 * hkv, D, generator=torch.Generator(device="cuda").manual_seed(B), device="cuda").to(BF)
    q[:, :2] = float("nan")                              # kv-head 0: all NaN
    words = summary_rows(s, hkv, D)[1]
    assert np.shares_memory(words, s)
    w = words.copy().view(np.uint16)                     # [pages, hkv, 2]
    w[:, 1, 0] = 0x7C00                                  # kv-head 1: infinite scales: infinities of either sign, or NaN
    w[:, 2, 1] = 0x7E00                                  # kv-head 2: zeros that are NaN
    words[:] = w.view(np.uint8)
    with np.errstate(all="ignore"):
        got = check(q, s, t, pages, lens, hkv, 16, True, 64, 140, 1, 2, False)
    assert (got[1][:, 0, :138] == np.arange(138)).all() and (got[1][:, 2, :138] == np.arange(138)).all()


@pytest.mark.parametrize("meta", [False, True])
@pytest.mark.parametrize("D,hq,hkv,h,L,take", [(64, 4, 2, 64, 9000, 60), (128, 8, 2, 128, 20000, 128), (128, 8, 1, 0, 6000, 40),
                                               (256, 6, 2, 256, 8000, 100)])
def test_lists_by_the_unrounded_scores(D, hq, hkv, h, L, take, meta):
    """q' . mean in 64 bits, q' not rounded to 8 bits: no page that is left out has a score above that of a page
    taken by more than twice what the rounding can do.  |q'_d - qs m_d| is at most qs / 2 (and the roundings of
    qs and its reciprocal: 127 qs 2^-22 at most), so a score moves by at most qs (1/2 + 2^-15) sum_d |mean_d|;
    three binary32 steps on partial values of at most qs (15 s + |z|) 127 D add less than 2^-22 of them."""
    lens = [L, L - 777]
    first, last = 2, 3
    q, s, bt, pages = make(D + hq, lens, hq, hkv, D, 16, BF, meta)
    got, st = run(q, s, bt, lens, hkv, 16, pages, h > 0, h or 16, take, first, last, meta)
    assert st == 0
    codes, words = summary_rows(s, hkv, D)
    n = np.empty((pages, hkv, D))
    n[..., 0::2], n[..., 1::2] = codes & 15, codes >> 4
    w = word_value(words.copy().view(np.uint16), meta).astype(np.float64)
    mean = n * w[..., :1] + w[..., 1:]
    x = q.double().cpu().numpy()
    if h:
        x = x @ matrix(h, D)
    for b, length in enumerate(lens):
        count = -(-length // 16)
        scored = np.arange(first, count - last)
        for k in range(hkv):
            G = hq // hkv
            y, m = x[b, k * G:(k + 1) * G], mean[bt[b, scored], k]
            score = (y @ m.T).max(0)
            qs = np.abs(y).max(-1) / 127
            s1, z1 = w[bt[b, scored], k, 0], np.abs(w[bt[b, scored], k, 1])
            slack = qs.max() * ((0.5 + 2.0 ** -15) * np.abs(m).sum(-1) + 2.0 ** -22 * 127 * D * (15 * s1 + z1))
            taken = np.isin(scored, got[1][b, k])
            assert taken.sum() == take - first - last
            assert (score - slack)[~taken].max() <= (score + slack)[taken].min()
