"""The serving-step calls at the sizes where offsets and counts grow: caches
beyond 2^32 bytes, more (sequence, kv-head) pairs than a workspace's shared
counter region, hundreds of groups, two captured steps on one workspace."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
import test_gpu_prefix as base
from gpu_helpers import ATTN_TOL, rel_err
from test_gpu_prefix import SEPARATE, SHARE
from test_gpu_rope import make

pytestmark = pytest.mark.gpu


def far_copy(small, page_bytes, far):
    """A cache of `far` pages more (left as they come), then the small one's."""
    big = torch.empty(far * page_bytes + small.numel(), dtype=torch.uint8, device="cuda")
    big[far * page_bytes:] = small
    return big


def test_prefix_decode_in_a_cache_beyond_32_bits():
    """The same pages 5.2 GB further on: the same bytes."""
    P, hkv, far = 64, 8, 150000
    s = base.setup(41, [30, 5], [512, 256], np.arange(35) * 7, hq=32, hkv=hkv, P=P)
    page = hkv * P * 68
    assert far * page > 2 ** 32
    t = dict(s, kc=far_copy(s["kc"], page, far), vc=far_copy(s["vc"], page, far), pages=s["pages"] + far,
             bt=np.where(s["bt"] >= 0, s["bt"] + far, -1))
    for mode in (SHARE, SEPARATE):
        (a, st), (b, st2) = base.run(s, mode=mode), base.run(t, mode=mode)
        assert st == st2 == 0 and torch.equal(a, b)


@pytest.mark.parametrize("T", [40, 3000])
def test_rope_append_in_a_cache_beyond_32_bits(T):
    P, hkv, far = 64, 8, 150000
    page = hkv * P * 68
    q, k, v, pages, slots, pos, cs = make(T, T, 16, hkv, 128, P, 128, torch.bfloat16)
    zero = torch.zeros(saw.saw_cache_bytes(pages, P, hkv, 128), dtype=torch.uint8, device="cuda")
    got = []
    for off in (0, far):
        kc, vc = far_copy(zero, page, off), far_copy(zero, page, off)
        qo, st = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
        saw.saw_rope_append(q, k, v, pos, cs, slots + off * P, qo, kc, vc, pages + off, P, True, True, 128, dev_status=st)
        assert st.item() == 0
        got.append((qo, kc[off * page:], vc[off * page:]))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_more_pairs_than_the_shared_counter_region():
    """17000 sequences by 8 kv-heads, next to a small batch on the same workspace."""
    s = base.setup(42, [16990, 10], [64, 32], np.random.default_rng(0).integers(0, 17, 17000), hq=8, hkv=8)
    ref = base.reference(s)
    need = saw.saw_prefix_decode_workspace_bytes(17000, 2, 8, 8, 128, 16, s["max_pre"], s["max_own"], SHARE)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for mode in (SHARE, SEPARATE):
        out, st = base.run(s, ws=ws, mode=mode)
        assert st == 0 and rel_err(out.cpu().numpy().reshape(-1, 128), ref, f"pairs-{mode}") <= ATTN_TOL


def test_hundreds_of_groups():
    """700 groups of one to three sequences, some without a prefix, a bad one among them."""
    rng = np.random.default_rng(5)
    sizes = rng.integers(1, 4, 700).tolist()
    pre = (rng.integers(0, 12, 700) * 16).tolist()
    pre[350], sizes[350] = 64, 2
    s = base.setup(43, sizes, pre, rng.integers(1, 60, sum(sizes)), hq=8, hkv=2)
    base.check(s, "700-groups")
    first = int(s["cu"][350])
    ref = base.reference(s).reshape(-1, 8, 128)
    s["pre"][350] = 10 ** 6
    rows = np.ones(sum(sizes), bool)
    rows[first:first + 2] = s["lens"][first:first + 2] <= s["max_own"]  # (its rows share nothing now)
    for mode in (SHARE, SEPARATE):
        out, st = base.run(s, mode=mode)
        assert st == saw.SAW_ERR_DEVICE_INDEX
        assert rel_err(out.cpu().numpy()[rows], ref[rows], f"700-bad-{mode}") <= ATTN_TOL


def test_two_graphs_and_eager_calls_on_one_workspace():
    """Two captured steps of different batches, replayed in turn with eager calls between, all on one workspace."""
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
    cases = [base.setup(44, [40], [1024], np.arange(40) * 30, hq=16, hkv=4),
             base.setup(45, [6, 3], [640, 256], np.arange(9) * 700, hq=16, hkv=4)]
    want = [base.run(s)[0] for s in cases]
    size = [saw.saw_prefix_decode_workspace_bytes(len(s["lens"]), len(s["pre"]), 16, 4, 128, 16, s["max_pre"],
                                                  s["max_own"], SHARE) for s in cases]
    ws = torch.zeros(max(size), dtype=torch.uint8, device="cuda")
    graphs, outs, keep = [], [], []
    for s in cases:
        args, out, graph = [i32(s[k]) for k in ("bt", "lens", "cu", "pre")], torch.empty_like(want[len(outs)]), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            saw.saw_prefix_decode_int4(s["q"], s["kc"], s["vc"], *args, s["max_pre"], s["max_own"], 4, s["pages"], 16, True,
                                       True, 128, out, ws, mode=SHARE)
        graphs.append(graph)
        outs.append(out)
        keep.append(args)
    for i in range(6):
        outs[i % 2].fill_(float("nan"))
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i % 2], want[i % 2])
        if i % 3 == 2:
            assert torch.equal(base.run(cases[i % 2], ws=ws)[0], want[i % 2])
