"""saw_prefix_decode_int4 where its arithmetic and its work list can go wrong:
scores far below zero, unreadable pages at the start of a part, faint keys,
lengths and groups that are refused next to good ones, own parts split over
CTAs behind a prefix.

Bar, where no other is derived at the test: the decode's, 2e-3 of the largest
output against the oracle's float64.
"""
import math

import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
import test_gpu_prefix as base
from gpu_helpers import ATTN_TOL, rel_err
from test_gpu_prefix import AUTO, SEPARATE, SHARE

pytestmark = pytest.mark.gpu


def append_rows(s, k=None, v=None):
    """Overwrite every slot's K rows, or V rows, or both: k, v float [slots] (the row's 128 values alike)."""
    wl, n = s["wl"], s["pages"] * s["wl"].page_size
    for cache, x, rot in (("kc", k, wl.rotate_k), ("vc", v, wl.rotate_v)):
        if x is not None:
            rows = torch.as_tensor(x, device="cuda").bfloat16()[:, None, None].expand(n, wl.num_kv_heads, 128)
            saw.saw_quantize_append(rows.contiguous(), None, torch.arange(n, device="cuda", dtype=torch.int32), s[cache],
                                    None, s["pages"], wl.page_size, rot, False, wl.block_h)


def slot_of(s, b, token):
    P = s["wl"].page_size
    return int(s["bt"][b, token // P]) * P + token % P


def steps_down(s, seed, top, by, levels=16):
    """Every slot's K row alike, and q all ones: scores -top, -(top + by), .. (natural, at sm_scale 1)."""
    i = np.random.default_rng(seed).integers(0, levels, s["pages"] * s["wl"].page_size)
    append_rows(s, k=-(top + by * i) / 128.0)
    s["q"] = torch.ones_like(s["q"])


@pytest.mark.parametrize("top", [32.0, 96.0, 128.0, 1024.0])
def test_scores_far_below_zero(top):
    """Every score of every tile is far below zero, past the exponents of binary32."""
    s = base.setup(31, [40, 7], [1024, 384], np.arange(47) % 30 + 1, rk=False)
    steps_down(s, 1, top, 2.0)
    base.check(s, f"below-{top}", sm_scale=1.0)


@pytest.mark.parametrize("P", [64, 16])
@pytest.mark.parametrize("top", [32.0, 128.0])
@pytest.mark.parametrize("bad", [(0,), (0, 1), (0, 1, 2, 3, 4), (1,), (0, 2, 7), tuple(range(1, 8)), tuple(range(8))])
def test_unreadable_tiles(P, top, bad):
    """Tiles of 128 keys with no valid page id, at a part's start and elsewhere: their keys do not count, the others
    do.  128 kv-heads: one part of all eight tiles each."""
    own = np.array([5, 40, 17])
    s = base.setup(32, [3], [1024], own, hq=128, hkv=128, P=P, rk=False)
    steps_down(s, 2, top, 2.0)
    per = 128 // P
    gone = [t * per + i for t in bad for i in range(per)]
    bt = s["bt"].copy()
    bt[:, gone] = -1
    out, st = base.run(dict(s, bt=bt), sm_scale=1.0)
    keep = [e for e in range(bt.shape[1]) if e not in gone]
    ref_bt = np.full_like(bt, -1)
    ref_bt[:, :len(keep)] = s["bt"][:, keep]
    ref = base.reference(s, sm_scale=1.0, bt=ref_bt, lens=s["lens"] - P * len(gone))
    assert st == saw.SAW_ERR_DEVICE_INDEX
    assert rel_err(out.cpu().numpy().reshape(-1, 128), ref, f"unreadable-{P}-{bad}") <= ATTN_TOL


def test_faint_keys_count():
    """One key of weight 1 and value 0, and n of weight w = 2^-25.2 and value 1: the output is n w / (1 + n w).
    p is held as a binary16 of 2^7 times its weight, so a faint key is off by at most half a step of 2^-24, 2^-32 of
    the first key's weight; what else rounds (the score 25.2 to 2^-19, the exponential to 2^-22, binary32 sums of
    n / 16 terms at 2^-23 each) is below 2^-12 of the output together."""
    s = base.setup(33, [3], [4096], np.array([1, 1, 1]), hq=128, hkv=128, rk=False, rv=False)
    n = s["pages"] * 16
    k, v = np.full(n, -1.0), np.ones(n)
    k[slot_of(s, 0, 700)] = v[slot_of(s, 0, 700)] = 0.0
    append_rows(s, k, v)
    s["q"] = torch.ones_like(s["q"])
    out, st = base.run(s, sm_scale=25.2 * math.log(2) / 128)
    w = 4096 * 2.0 ** -25.2
    want = w / (1 + w)
    assert st == 0
    assert np.abs(out.double().cpu().numpy() - want).max() <= 4096 * 2.0 ** -32 + want * 2.0 ** -12


@pytest.mark.parametrize("length", [1 << 20, 512 + 200, 512 + 101, -3, 100])
def test_refused_rows_are_not_read_for_the_others(length):
    """A group's first sequence is refused for its length: its table row, which then may hold anything, is not the
    one that the prefix is read through."""
    s = base.setup(34, [20], [512], np.full(20, 100), hq=8, hkv=2)
    ref = base.reference(s).reshape(20, 8, 128)
    s["lens"][0] = length
    s["bt"][0] = np.random.default_rng(0).permutation(s["pages"])[:s["bt"].shape[1]]
    for mode in (SHARE, SEPARATE):
        out, st = base.run(s, mode=mode)
        assert st == saw.SAW_ERR_DEVICE_INDEX and (out[0] == 0).all()
        assert rel_err(out[1:].cpu().numpy(), ref[1:], f"refused-{length}") <= ATTN_TOL


@pytest.mark.parametrize("entry", [1000, 41, -5, 5, 25])
@pytest.mark.parametrize("generous", [False, True])
def test_a_bad_group_between_good_ones(entry, generous):
    """One wrong entry of cu_group_seqs: the groups it bounds share nothing, the others are as before."""
    s = base.setup(35, [10] * 4, [512, 256, 384, 320], np.full(40, 20), hq=8, hkv=2)
    ref = base.reference(s).reshape(40, 8, 128)
    s["cu"][2] = entry
    if generous:
        s["max_own"] = 512 + 20
    good = list(range(40)) if generous else list(range(10)) + list(range(30, 40))
    if entry == 25:  # in range: the second group takes rows of the third, whose prefix is another
        good = [b for b in good if not 20 <= b < 25]
    for mode in (SHARE, SEPARATE):
        out, st = base.run(s, mode=mode)
        assert st == saw.SAW_ERR_DEVICE_INDEX or entry == 25
        assert rel_err(out[good].cpu().numpy(), ref[good], f"bad-middle-{entry}") <= ATTN_TOL


SPLIT = [
    (6, 1, 2, 16, 5000, torch.float32), (6, 4, 2, 64, 9000, torch.bfloat16), (10, 8, 2, 32, 3000, torch.float32),
    (3, 7, 1, 16, 20000, torch.float32), (20, 4, 8, 16, 2500, torch.bfloat16),
]


@pytest.mark.parametrize("B,G,hkv,P,longest,dt", SPLIT)
def test_own_parts_split_over_ctas(B, G, hkv, P, longest, dt):
    """Own parts of several splits each behind shared prefixes: none, one token, and up to the longest; an idle row;
    two groups and a sequence in none."""
    own = np.random.default_rng(B).integers(1, longest, B)
    own[:3] = longest, 0, 1
    s = base.setup(B, [B - 1, 1], [640, 192], own, hq=G * hkv, hkv=hkv, P=P)
    assert saw.saw_decode_plan(B, hkv, P, s["max_own"])[0] > 1
    base.check(s, f"split-{B}-{G}-{P}", dt)
    s["cu"], s["pre"] = s["cu"][:2], s["pre"][:1]
    s["lens"][1] = 0
    base.check(s, f"split-idle-{B}-{G}-{P}", dt)


@pytest.mark.parametrize("mode", [SHARE, SEPARATE])
def test_split_own_parts_repeat_bit_for_bit(mode):
    """Whichever split of a sequence ends last, the same sum: 200 calls, one result."""
    s = base.setup(37, [8], [1024], np.random.default_rng(3).integers(2000, 9000, 8), hq=8, hkv=2)
    assert saw.saw_decode_plan(8, 2, 16, s["max_own"])[0] > 2
    need = saw.saw_prefix_decode_workspace_bytes(8, 1, 8, 2, 128, 16, s["max_pre"], s["max_own"], mode)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first, st = base.run(s, ws=ws, mode=mode)
    assert st == 0
    differ = sum(not torch.equal(base.run(s, ws=ws, mode=mode)[0], first) for _ in range(200))
    assert differ == 0


@pytest.mark.parametrize("rk", [True, False])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_nan_queries_stay_nan(rk, dt):
    """A NaN in a head's q makes that row of the output NaN, as the plain decode does, and no other."""
    s = base.setup(38, [30], [768], np.arange(30) % 3 * 20, hq=8, hkv=2, rk=rk, dt=dt)
    ref = base.reference(s).reshape(30, 8, 128)
    s["q"] = s["q"].clone()
    rows = [(0, 0, 0), (7, 3, 127), (9, 7, 64), (29, 5, 1)]
    bad = torch.zeros(30, 8, dtype=torch.bool)
    for b, h, d in rows:
        s["q"][b, h, d] = float("nan")
        bad[b, h] = True
    for mode in (SHARE, SEPARATE):
        out, st = base.run(s, mode=mode)
        out = out.cpu()
        assert st == 0 and out[bad].isnan().all()
        assert rel_err(out[~bad].numpy(), ref[~bad.numpy()], f"nan-{mode}") <= ATTN_TOL


@pytest.mark.parametrize("tokens,groups", [(128, 1), (128, 150), (64, 400)])
def test_parts_of_one_tile(tokens, groups):
    """Parts of a single tile, one and many to a CTA: one set of softmax warps has nothing to do but the part's end.
    Every call of two hundred gives the same bits."""
    B = 2 * groups
    s = base.setup(46, [2] * groups, [tokens] * groups, np.arange(B) % 5 * 3, hq=16, hkv=4)
    base.check(s, f"one-tile-{tokens}x{groups}")
    need = saw.saw_prefix_decode_workspace_bytes(B, groups, 16, 4, 128, 16, s["max_pre"], s["max_own"], SHARE)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first, _ = base.run(s, ws=ws)
    assert all(torch.equal(base.run(s, ws=ws)[0], first) for _ in range(200))
