"""saw_prefix_decode_int4 against the oracle's float64 decode of every
sequence over its own whole table (the definition: sharing changes nothing
but what is read).

Bar: max |o - o_ref| / max |o_ref| <= 2e-3 for a float32 output, the
decode's.  The prefix pass takes K's codes exactly and q in two binary16
parts; it rounds the dequantized V and p to binary16 once each, at most 2^-11
of each value and 2^-12 on average, in a weighted mean of V: below 2^-10 of the
largest V.  A 16-bit output adds its one rounding, at most half a step of the
value: 2^-8 or 2^-11.
"""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from bit_paged_kv_gb300 import workloads as W
from gpu_helpers import ATTN_TOL, new_caches, oracle_decode, rel_err

pytestmark = pytest.mark.gpu


def setup(seed, sizes, pre, own, hq=8, hkv=2, P=16, rk=True, rv=True, h=128, dt=torch.bfloat16, meta=False,
          spare=5, dist="student_t", extra_blocks=1):
    """sizes: sequences per group; pre: shared tokens per group (whole pages are shared);
    own: tokens behind the whole pages of the prefix, per sequence."""
    wl = W.TINY.variant(num_q_heads=hq, num_kv_heads=hkv, page_size=P, rotate_k=rk, rotate_v=rv, block_h=h,
                        dist=dist, nu=4, seed=seed)
    B = sum(sizes)
    whole = [x // P * P for x in pre]
    of = np.repeat(np.arange(len(sizes)), sizes)
    lens = np.array([whole[of[b]] + own[b] for b in range(B)], np.int64)
    blocks = max(max(-(-int(n) // P) for n in lens), max(whole) // P, 1) + extra_blocks
    n_pages = sum(w // P for w in whole) + sum(-(-int(o) // P) for o in own) + spare
    ids = np.random.default_rng(seed).permutation(n_pages)
    bt = np.full((B, blocks), -1, np.int32)
    at = 0
    for g, w in enumerate(whole):
        bt[of == g, :w // P] = ids[at:at + w // P]
        at += w // P
    for b in range(B):
        a, m = whole[of[b]] // P, -(-int(own[b]) // P)
        bt[b, a:a + m] = ids[at:at + m]
        at += m
    k = W.kv_rows(wl, 0, W.K, n_pages * P, "cuda", dtype=dt)
    v = W.kv_rows(wl, 0, W.V, n_pages * P, "cuda", dtype=dt)
    kc, vc = new_caches(n_pages, P, hkv, 128)
    saw.saw_quantize_append(k, v, torch.arange(n_pages * P, device="cuda", dtype=torch.int32), kc, vc, n_pages, P,
                            rk, rv, h, meta_bf16=meta)
    q = W.q_rows(wl, 0, "cuda", num_seqs=B, dtype=dt)
    cu = np.concatenate(([0], np.cumsum(sizes)))
    return dict(wl=wl, q=q, kc=kc, vc=vc, bt=bt, lens=lens, cu=cu, pre=np.array(pre), pages=n_pages, meta=meta,
                max_pre=int(max(pre)), max_own=int(max(list(own) + [0])))


SHARE, SEPARATE, AUTO = saw.SAW_PREFIX_SHARE, saw.SAW_PREFIX_SEPARATE, saw.SAW_PREFIX_AUTO


def run(s, out_dtype=torch.float32, sm_scale=0.0, ws=None, stream=None, mode=SHARE, **kw):
    s = dict(s, **kw)
    wl, q = s["wl"], s["q"]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    B, G = q.shape[0], len(s["pre"])
    out = torch.full(q.shape, float("nan"), dtype=out_dtype, device="cuda")
    need = saw.saw_prefix_decode_workspace_bytes(B, G, wl.num_q_heads, wl.num_kv_heads, 128, wl.page_size,
                                                 s["max_pre"], s["max_own"], mode)
    if ws is None:
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    assert ws.numel() >= need
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = [i32(s[k]) for k in ("bt", "lens", "cu", "pre")]
    torch.cuda.synchronize()
    saw.saw_prefix_decode_int4(q, s["kc"], s["vc"], *args, s["max_pre"], s["max_own"], wl.num_kv_heads, s["pages"],
                               wl.page_size, wl.rotate_k, wl.rotate_v, wl.block_h, out, ws, sm_scale=sm_scale,
                               dev_status=st, meta_bf16=s["meta"], stream=stream, mode=mode)
    torch.cuda.synchronize()
    return out, int(st.item())


def reference(s, sm_scale=None, bt=None, lens=None):
    wl = s["wl"]
    return oracle_decode(s["q"], s["kc"].cpu().numpy(), s["vc"].cpu().numpy(),
                         torch.from_numpy(s["bt"] if bt is None else bt),
                         torch.from_numpy((s["lens"] if lens is None else lens).astype(np.int32)), wl.num_kv_heads,
                         s["pages"], wl.page_size, wl.rotate_k, wl.rotate_v, wl.block_h, sm_scale=sm_scale,
                         meta_bf16=s["meta"])


def check(s, label, out_dtype=torch.float32, sm_scale=0.0):
    ref = reference(s, sm_scale or None)
    tol = ATTN_TOL + (0 if out_dtype is torch.float32 else torch.finfo(out_dtype).eps / 2)
    for mode in (SEPARATE, AUTO, SHARE):
        out, st = run(s, out_dtype, sm_scale, mode=mode)
        assert st == 0
        got = out.float().cpu().numpy().reshape(-1, 128)
        assert np.isfinite(got).all()
        err = rel_err(got, ref, f"prefix-{label}")
        assert err <= tol, f"mode {mode}: relative error {err:.3e}"
    return out


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("P", [16, 32, 64])
def test_groups_of_heads(G, P):
    rng = np.random.default_rng(G * 100 + P)
    s = setup(G + P, [21], [640 + P], rng.integers(1, 90, 21), hq=2 * G, hkv=2, P=P)
    check(s, f"G{G}-P{P}")


@pytest.mark.parametrize("sizes,pre", [
    ([40], [16]), ([40], [128]), ([40], [144]), ([33], [2000]), ([64], [4096]), ([70, 3, 1, 30], [300, 0, 512, 1024]),
    ([1, 90], [700, 700]), ([40, 0, 40], [256, 256, 272]), ([130], [513]), ([300], [272]), ([17] * 9, [160] * 9),
    ([3] * 40, [48 * i for i in range(40)]),
])
def test_batches(sizes, pre):
    rng = np.random.default_rng(len(sizes) * 1000 + pre[0])
    check(setup(7, sizes, pre, rng.integers(1, 200, sum(sizes)), hq=8, hkv=2), f"{len(sizes)}x{pre[0]}")


@pytest.mark.parametrize("rk,rv,h", [(1, 1, 128), (1, 0, 128), (0, 0, 128), (0, 1, 64), (1, 1, 64), (1, 0, 32), (1, 1, 16)])
@pytest.mark.parametrize("dt,meta", [(torch.bfloat16, True), (torch.float16, False)])
def test_rotations_and_formats(rk, rv, h, dt, meta):
    rng = np.random.default_rng(h)
    s = setup(3, [50], [1000], rng.integers(1, 70, 50), hq=16, hkv=4, P=32, rk=bool(rk), rv=bool(rv), h=h, dt=dt,
              meta=meta)
    check(s, f"{rk}{rv}-h{h}")
    check(s, f"{rk}{rv}-h{h}-out16", out_dtype=dt)


def test_the_serving_shapes():
    """32 and 64 q-heads over 8, a longer prefix, 16-bit output; own parts of one token to several splits."""
    rng = np.random.default_rng(1)
    own = rng.integers(1, 300, 64)
    own[5], own[6] = 1, 3000
    check(setup(1, [64], [8192], own, hq=32, hkv=8), "64x8192", torch.bfloat16)
    check(setup(2, [96], [1024], rng.integers(1, 40, 96), hq=64, hkv=8), "96x1024", torch.bfloat16)


def test_sequences_that_end_with_the_prefix_and_idle_rows():
    own = np.array([0, 5, 0, 30, 17] * 9)
    s = setup(5, [45], [336], own, hq=8, hkv=2)
    s["lens"][7] = s["lens"][20] = 0
    out = check(s, "empty-own")
    assert (out[7] == 0).all() and (out[20] == 0).all()


@pytest.mark.parametrize("G,P", [(8, 16), (4, 64), (3, 32)])
def test_many_sequences(G, P):
    """More (sequence, kv-head) pairs than four per SM: the second pass in its smallest CTAs, own parts from nothing
    to many turns of their rings, an unreadable page in one of them."""
    rng = np.random.default_rng(G)
    own = rng.integers(0, 900, 320)
    own[:4] = 0, 1, 63, 64
    s = setup(24, [300, 20], [256, 64], own, hq=2 * G, hkv=2, P=P)
    check(s, f"many-G{G}-P{P}")
    b = int(np.argmax(own[:300]))
    bt, e = s["bt"].copy(), 256 // P + 1
    bt[b, e] = -1
    out, st = run(dict(s, bt=bt))
    keep = [i for i in range(bt.shape[1]) if i != e]
    ref = reference(s, bt=np.where(np.arange(320)[:, None] == b, np.pad(s["bt"][:, keep], ((0, 0), (0, 1))), s["bt"]),
                    lens=np.where(np.arange(320) == b, s["lens"] - P, s["lens"]))
    assert st == saw.SAW_ERR_DEVICE_INDEX
    assert rel_err(out.cpu().numpy().reshape(-1, 128), ref, f"many-bad-G{G}-P{P}") <= ATTN_TOL


def test_nothing_behind_the_prefix():
    """Every sequence ends with its prefix: max_own_len 0."""
    check(setup(23, [40, 3], [512, 128], [0] * 43, hq=8, hkv=2), "no-own")


def test_idle_rows_may_hold_anything_in_their_tables():
    """Groups whose first sequences (more than a warp's lanes of them), or all, are idle, with no page in their
    table rows: as if they were not there."""
    for sizes, idle in (([12], [0]), ([50], list(range(40))), ([6, 5, 9], [0, 1, 6, 7, 8, 9, 10, 19])):
        s = setup(21, sizes, [272, 400, 160][:len(sizes)], np.arange(1, sum(sizes) + 1), hq=8, hkv=2)
        s["lens"][idle] = 0
        s["bt"][idle] = -1
        out = check(s, "idle-first")
        assert (out[idle] == 0).all()


def test_bad_group_behind_many_is_reported():
    s = setup(22, [2] * 40, [32] * 40, np.arange(1, 81), hq=8, hkv=2)
    s["cu"], s["pre"] = np.append(s["cu"], 80), np.append(s["pre"], -1)
    want = reference(s).reshape(80, 8, 128)
    for mode in (SHARE, SEPARATE):
        out, st = run(s, mode=mode)
        assert st == saw.SAW_ERR_DEVICE_INDEX and rel_err(out.cpu().numpy(), want, "prefix-bad-last") <= ATTN_TOL


def test_one_sequence_and_one_token():
    check(setup(6, [1], [400], [1]), "single")
    check(setup(6, [2], [0], [1, 1]), "no-prefix")
    check(setup(6, [1, 1], [16, 32], [0, 1]), "two")


def test_part_of_a_page_is_read_per_sequence():
    """prefix_lens inside a page: the whole pages are shared, the rest is each sequence's own."""
    s = setup(8, [50], [16 * 40], np.arange(1, 51), hq=8, hkv=2, P=64)
    s["pre"] = s["pre"] + 63
    s["max_pre"] += 63
    check(s, "in-page")


def test_ungrouped_sequences():
    """Sequences before, between and behind the groups share nothing."""
    s = setup(9, [5, 40, 6], [64, 256, 64], np.arange(1, 52), hq=8, hkv=2)
    s["cu"], s["pre"] = np.array([5, 45]), np.array([256])
    s["max_own"] = int(s["lens"].max())
    check(s, "ungrouped")
    s["cu"], s["pre"], s["max_pre"] = np.array([0]), np.zeros(0, int), 0
    check(s, "no-groups")


def test_scale_and_heavy_logits():
    s = setup(10, [40], [900], np.arange(1, 41), hq=8, hkv=2)
    check(s, "scale", sm_scale=0.5)
    check(s, "scale-small", sm_scale=1e-3)


def test_agrees_with_the_plain_decode():
    s = setup(11, [60], [1024], np.arange(1, 61), hq=32, hkv=8)
    out, st = run(s)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    L = int(s["lens"].max())
    ref = torch.empty_like(out)
    ws = torch.zeros(max(16, saw.saw_decode_workspace_bytes(60, 32, 8, 128, 16, L)), dtype=torch.uint8, device="cuda")
    saw.saw_paged_decode_int4(s["q"], s["kc"], s["vc"], i32(s["bt"]), i32(s["lens"]), L, 8, s["pages"], 16, True, True,
                              128, ref, ws)
    assert st == 0 and rel_err(out.cpu().numpy(), ref.cpu().numpy(), "prefix-vs-decode") <= ATTN_TOL


def test_bad_lengths_and_groups_are_reported():
    own = np.full(40, 20)
    s = setup(12, [20, 20], [256, 128], own, hq=8, hkv=2)
    want = reference(s).reshape(40, 8, 128)
    for what in ("short", "negative", "long", "cu", "prefix", "prefix_neg"):
        t = dict(s, lens=s["lens"].copy(), cu=s["cu"].copy(), pre=s["pre"].copy())
        bad = []
        if what == "short":
            t["lens"][3], bad = 200, [3]
        elif what == "negative":
            t["lens"][39], bad = -5, [39]
        elif what == "long":
            t["lens"][25], bad = 128 + 21, [25]
        elif what == "cu":
            t["cu"][2], t["max_own"] = 41, 300      # group 1 past the batch: shares nothing
        elif what == "prefix":
            t["pre"][1], t["max_own"] = 257, 300
        else:
            t["pre"][0], t["max_own"] = -1, 300
        for mode in (SHARE, SEPARATE):
            out, st = run(t, mode=mode)
            assert st == saw.SAW_ERR_DEVICE_INDEX, what
            got = out.cpu().numpy()
            ok = [b for b in range(40) if b not in bad]
            assert rel_err(got[ok], want[ok], f"prefix-bad-{what}") <= ATTN_TOL
            assert all((got[b] == 0).all() for b in bad)


def test_bad_pages_are_skipped():
    """Invalid ids in the prefix (the same in every row, as the prefix is) and one behind it: those keys
    do not count."""
    own = np.full(50, 40)
    s = setup(13, [50], [512], own, hq=8, hkv=2)
    bt = s["bt"].copy()
    bt[:, 3], bt[:, 9], bt[7, 33] = s["pages"], -1, s["pages"] + 1000
    out, st = run(dict(s, bt=bt))
    assert st == saw.SAW_ERR_DEVICE_INDEX
    ref_bt, lens = s["bt"].copy(), s["lens"] - 32
    keep = [i for i in range(34 + 1) if i not in (3, 9)]
    ref_bt[:, :len(keep)] = s["bt"][:, keep]
    ref_bt[7, 31:] = -1
    seven = [b for b in range(50) if b != 7]
    ref = reference(s, bt=ref_bt, lens=np.where(np.arange(50) == 7, 512 - 32 + 16, lens)).reshape(50, 8, 128)
    # sequence 7: prefix, own page 32, not 33; its last 8 tokens lie on page 34
    got = out.cpu().numpy()
    assert rel_err(got[seven], ref[seven], "prefix-bad-page") <= ATTN_TOL
    assert np.isfinite(got).all()


def test_keys_outside_the_sequences_do_not_matter():
    """Whatever lies on pages and rows no sequence reaches (infinities and NaN as scales): the same bytes out."""
    own = np.arange(1, 41)
    s = setup(14, [40], [16 * 21], own, hq=8, hkv=2)
    a, _ = run(s)
    used = np.zeros((s["pages"], 16), bool)
    for b in range(40):
        for t in range(int(s["lens"][b])):
            used[s["bt"][b, t // 16], t % 16] = True
    mask = torch.from_numpy(~used).cuda()
    for name in ("kc", "vc"):
        c = s[name].clone().view(s["pages"], 2, 1088)
        words = c[:, :, 1024:].view(torch.int16).view(s["pages"], 2, 16, 2)
        words[mask[:, None, :, None].expand_as(words)] = 0x7C00
        words[..., 1][mask[:, None].expand(s["pages"], 2, 16)] = 0x7E00
        s[name] = c.view(-1)
    b, st = run(s)
    assert st == 0 and torch.equal(a, b)


def test_repeated_calls_share_a_workspace():
    """A workspace serves call after call, of this shape and of smaller ones, and the answer does not change."""
    s = setup(15, [64], [2048], np.arange(1, 65) * 20, hq=32, hkv=8)
    need = saw.saw_prefix_decode_workspace_bytes(64, 1, 32, 8, 128, 16, s["max_pre"], s["max_own"], SHARE)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first, _ = run(s, ws=ws)
    small = setup(16, [8], [512], np.arange(1, 9), hq=32, hkv=8)
    alone, _ = run(small)
    for _ in range(3):
        again, st = run(s, ws=ws)
        assert st == 0 and torch.equal(first, again)
        other, st = run(small, ws=ws)
        assert st == 0 and torch.equal(other, alone)
    many = setup(19, [100] * 3, [160] * 3, np.arange(1, 301) * 8, hq=32, hkv=8)
    need = max(need, saw.saw_prefix_decode_workspace_bytes(300, 3, 32, 8, 128, 16, 160, many["max_own"], SHARE))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    alone, _ = run(many)
    for _ in range(2):
        assert torch.equal(run(many, ws=ws)[0], alone) and torch.equal(run(s, ws=ws)[0], first)


def test_graph_replay_with_new_inputs_and_other_stream():
    s = setup(17, [48], [1024], np.arange(1, 49), hq=32, hkv=8)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a, _ = run(s)
    b, _ = run(s, stream=side)
    assert torch.equal(a, b)
    wl = s["wl"]
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    args = [i32(s[k]) for k in ("bt", "lens", "cu", "pre")]
    need = saw.saw_prefix_decode_workspace_bytes(48, 1, 32, 8, 128, 16, s["max_pre"], s["max_own"], SHARE)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    out = torch.empty(s["q"].shape, device="cuda")
    q = s["q"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            saw.saw_prefix_decode_int4(q, s["kc"], s["vc"], *args, s["max_pre"], s["max_own"], 8, s["pages"], 16, True,
                                       True, 128, out, ws, mode=SHARE)
    q.copy_(s["q"].flip(0))
    lens = s["lens"].copy()
    lens[::3] = 1024 + 1
    args[1].copy_(i32(lens))
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    t = dict(s, q=q, lens=lens)
    assert rel_err(out.cpu().numpy().reshape(-1, 128), reference(t), "prefix-graph") <= ATTN_TOL


def test_two_streams_at_once():
    """Calls of different batches in flight on two streams, each with its own workspace."""
    i32 = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()
    sides = []
    for seed, B, pre in ((25, 64, 2048), (26, 90, 800)):
        s = setup(seed, [B], [pre], np.arange(1, B + 1) * 9, hq=32, hkv=8)
        need = saw.saw_prefix_decode_workspace_bytes(B, 1, 32, 8, 128, 16, pre, s["max_own"], SHARE)
        sides.append(dict(s=s, want=run(s)[0], args=[i32(s[k]) for k in ("bt", "lens", "cu", "pre")],
                          ws=torch.zeros(need, dtype=torch.uint8, device="cuda"), stream=torch.cuda.Stream(),
                          outs=[torch.empty(s["q"].shape, device="cuda") for _ in range(8)]))
    torch.cuda.synchronize()
    for i in range(8):
        for x in sides:
            s = x["s"]
            saw.saw_prefix_decode_int4(s["q"], s["kc"], s["vc"], *x["args"], s["max_pre"], s["max_own"], 8, s["pages"],
                                       16, True, True, 128, x["outs"][i], x["ws"], stream=x["stream"], mode=SHARE)
    torch.cuda.synchronize()
    for x in sides:
        assert all(torch.equal(o, x["want"]) for o in x["outs"])


def test_long_prefix():
    """One 100000-token prefix, page 64: offsets, many partials per row."""
    s = setup(18, [24], [100032], np.arange(1, 25) * 3, hq=8, hkv=2, P=64)
    check(s, "long", torch.bfloat16)
