"""The sparse decode step's calls at the far end: caches and summaries beyond 2^32
bytes, the same pages at their start and behind 4 GiB giving the same bytes; many
sequences; two calls at once on two streams."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from sparse_oracle import summary_stride

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HKV, D, P = 8, 128, 16
CHUNK = HKV * P * (D // 2 + 4)


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def test_caches_beyond_4_gib():
    """Normed append, summaries and decode with page ids behind 2^32 bytes."""
    pages = 2 ** 32 // CHUNK + 200
    T, shift = 40 * P, pages - 50
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda").to(BF) for h in (32, HKV, HKV))
    w = (1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")).to(BF)
    cs = torch.empty(1024, D, device="cuda")
    saw.saw_rope_table(cs, 1e6)
    pos = torch.arange(T, device="cuda").int()
    status, got = i32([0]), []
    big = [torch.zeros(pages * CHUNK, dtype=torch.uint8, device="cuda") for _ in range(2)]
    assert big[0].numel() > 2 ** 32 and shift * CHUNK > 2 ** 32
    lists = torch.stack([torch.randperm(40, generator=torch.Generator().manual_seed(i))[:24] for i in range(HKV)]).int().cuda()[None]
    for first in (0, shift):
        slots = (torch.arange(T, device="cuda") + first * P).int()
        qo = torch.empty_like(q)
        saw.saw_norm_rope_append(q, k, v, w[0], w[1], pos, cs, slots, qo, *big, pages, P, True, True, 128, dev_status=status)
        summary = torch.zeros(saw.saw_summary_bytes(pages, HKV, D), dtype=torch.uint8, device="cuda")
        bt = (torch.arange(40, device="cuda") + first).int()[None].contiguous()
        saw.saw_page_summary(big[0], bt, i32([T]), None, T, HKV, D, pages, P, summary, dev_status=status)
        out = torch.empty(1, 32, D, dtype=BF, device="cuda")
        need = saw.saw_sparse_decode_workspace_bytes(1, 32, HKV, D, P, 24 * P)
        ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
        saw.saw_sparse_decode_int4(qo[-1:].contiguous(), *big, lists + first, torch.full((1, HKV), 24 * P - 3, dtype=torch.int32, device="cuda"),
                                   24 * P, HKV, pages, P, True, True, 128, out, ws, dev_status=status)
        rows = summary.view(pages, -1)[first:first + 40]
        got.append((qo, *(x.view(pages, -1)[first:first + 40].clone() for x in big), rows.clone(), out))
    assert status.item() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.float().abs().sum() > 0


@pytest.mark.parametrize("B", [1, 70])
def test_summaries_beyond_4_gib(B):
    stride = summary_stride(HKV, D)
    pages = 2 ** 32 // stride + 3000
    rng = np.random.default_rng(B)
    near = torch.from_numpy(rng.integers(0, 256, (2000, stride), dtype=np.uint8)).cuda()
    # (finite words: scales and zeros of small exponents)
    near[:, HKV * D // 2:HKV * (D // 2 + 4)] &= 0x3B
    far = torch.zeros(pages * stride, dtype=torch.uint8, device="cuda")
    assert far.numel() > 2 ** 32
    shift = pages - 2000
    far.view(pages, stride)[shift:] = near
    lens = rng.integers(900, 1999 * P // max(1, B // 4), B)
    need = -(-lens // P)
    bt = np.stack([rng.permutation(2000)[:need.max()] for _ in range(B)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((B, 32, D)).astype(np.float32)).to(BF).cuda()
    out = []
    for s, n, add in ((near.view(-1), 2000, 0), (far, pages, shift)):
        tables, nos, sl = (torch.zeros(z, dtype=torch.int32, device="cuda") for z in ((B, HKV, 30), (B, HKV, 30), (B, HKV)))
        st = i32([0])
        saw.saw_select_pages(q, s, i32(bt + add), i32(lens), int(lens.max()), HKV, n, P, True, 128, 1, 2, tables, sl,
                             sel_pages=nos, dev_status=st)
        assert st.item() == 0
        out.append((tables - add, nos, sl))
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_most_sequences():
    """65535 sequences of a page or two: one grid row each."""
    B, hkv, d = 65535, 1, 64
    pages = 64
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(pages * P, hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
    kc, vc = (torch.zeros(saw.saw_cache_bytes(pages, P, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    saw.saw_quantize_append(k, v, torch.arange(pages * P, device="cuda").int(), kc, vc, pages, P, True, True, 64)
    bt = torch.randint(0, pages, (B, 4), generator=g, device="cuda").int()
    lens = torch.randint(0, 65, (B,), generator=g, device="cuda").int()
    summary = torch.zeros(saw.saw_summary_bytes(pages, hkv, d), dtype=torch.uint8, device="cuda")
    st = i32([0])
    saw.saw_page_summary(kc, bt, lens, None, 64, hkv, d, pages, P, summary, dev_status=st)
    q = torch.randn(B, 2, d, generator=g, device="cuda").to(BF)
    tables, nos, sl = (torch.zeros(z, dtype=torch.int32, device="cuda") for z in ((B, hkv, 3), (B, hkv, 3), (B, hkv)))
    saw.saw_select_pages(q, summary, bt, lens, 64, hkv, pages, P, True, 64, 1, 1, tables, sl, sel_pages=nos, dev_status=st)
    out = torch.empty_like(q)
    need = saw.saw_sparse_decode_workspace_bytes(B, 2, hkv, d, P, 48)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device="cuda")
    saw.saw_sparse_decode_int4(q, kc, vc, tables, sl, 48, hkv, pages, P, True, True, 64, out, ws, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    n = (lens + P - 1) // P
    want = torch.where(n > 3, lens - P, lens)
    assert torch.equal(sl[:, 0], want) and torch.equal((nos[:, 0] >= 0).sum(-1), n.clamp(max=3).long())
    # the same sequences alone
    for b in (0, 1, 777, 40000, B - 1):
        one = torch.empty(1, 2, d, dtype=BF, device="cuda")
        saw.saw_sparse_decode_int4(q[b:b + 1], kc, vc, tables[b:b + 1], sl[b:b + 1], 48, hkv, pages, P, True, True, 64, one, ws)
        # (another CTA shape adds its warps' parts in another order: a bfloat16 step, 2^-7 at most)
        tol = 2.0 ** -7 * out[b].float().abs() + 2.0 ** -12
        assert (out[b].float() - one[0].float()).abs().le(tol).all()


def test_two_streams():
    """Two steps' selections and decodes under way together, each with a workspace of its own."""
    g = torch.Generator(device="cuda").manual_seed(4)
    pages, B, take = 3000, 2, 300
    k, v = (torch.randn(pages * P, HKV, D, generator=g, device="cuda").to(BF) for _ in range(2))
    kc, vc = (torch.zeros(pages * CHUNK, dtype=torch.uint8, device="cuda") for _ in range(2))
    saw.saw_quantize_append(k, v, torch.arange(pages * P, device="cuda").int(), kc, vc, pages, P, True, True, 128)
    summary = torch.zeros(saw.saw_summary_bytes(pages, HKV, D), dtype=torch.uint8, device="cuda")
    lens = i32([20000, 17000])
    bt = torch.stack([torch.randperm(pages, generator=g, device="cuda")[:1250] for _ in range(B)]).int()
    saw.saw_page_summary(kc, bt, lens, None, 20000, HKV, D, pages, P, summary)
    need = saw.saw_sparse_decode_workspace_bytes(B, 32, HKV, D, P, take * P)
    assert need > 0
    jobs = []
    for i in range(2):
        jobs.append(dict(q=torch.randn(B, 32, D, generator=g, device="cuda").to(BF), out=torch.empty(B, 32, D, dtype=BF, device="cuda"),
                         ws=torch.zeros(need, dtype=torch.uint8, device="cuda"), s=torch.cuda.Stream(),
                         t=torch.zeros(B, HKV, take, dtype=torch.int32, device="cuda"),
                         l=torch.zeros(B, HKV, dtype=torch.int32, device="cuda"), st=i32([0])))

    def go(j):
        saw.saw_select_pages(j["q"], summary, bt, lens, 20000, HKV, pages, P, True, 128, 1, 4, j["t"], j["l"], dev_status=j["st"])
        saw.saw_sparse_decode_int4(j["q"], kc, vc, j["t"], j["l"], take * P, HKV, pages, P, True, True, 128, j["out"], j["ws"],
                                   dev_status=j["st"])

    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            with torch.cuda.stream(j["s"]):
                go(j)
    torch.cuda.synchronize()
    for j in jobs:
        got = j["out"].clone(), j["t"].clone()
        go(j)
        torch.cuda.synchronize()
        assert j["st"].item() == 0
        assert torch.equal(got[0], j["out"]) and torch.equal(got[1], j["t"])
