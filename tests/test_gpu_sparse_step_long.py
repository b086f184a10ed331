"""A sparse decode step over long prompts: lists that are split and merged, and a
selection by a cluster, in the chain of normed append, summaries, selection and
decode, eager and as one replayed graph.  Summaries and lists are checked byte for
byte from the caches and queries on the device, the attention in 64 bits."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from gpu_helpers import assert_bytes_equal
from sparse_oracle import attend, select, summaries

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,hq,hkv,prompts,take", [(128, 8, 2, [6000, 4321], 90), (64, 12, 2, [5000], 70),
                                                   (256, 4, 1, [4500, 4400, 900], 66)])
def test_split_lists_and_clusters(D, hq, hkv, prompts, take, odt):
    P, B, first, last, h, steps = 16, len(prompts), 1, 3, 64, 4
    blocks = [-(-(n + steps) // P) for n in prompts]
    assert max(blocks) > 256 and take * P > 1024
    pages = sum(blocks) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(D)).int()
    bt, at = torch.full((B, max(blocks)), -1, dtype=torch.int32), 0
    for b, n in enumerate(blocks):
        bt[b, :n] = order[at:at + n]
        at += n
    slot_of = [(bt[b, :n, None].long() * P + torch.arange(P)).flatten().int() for b, n in enumerate(blocks)]
    g = torch.Generator(device=DEV).manual_seed(D)
    qkv = lambda n: [torch.randn(n, x, D, generator=g, device=DEV).bfloat16() for x in (hq, hkv, hkv)]
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g, device=DEV)).bfloat16()
    cs = torch.empty(8192, D, device=DEV)
    saw.saw_rope_table(cs, 1e6)
    kc, vc = (torch.zeros(saw.saw_cache_bytes(pages, P, hkv, D), dtype=torch.uint8, device=DEV) for _ in range(2))
    summary = torch.full((saw.saw_summary_bytes(pages, hkv, D),), 0xAB, dtype=torch.uint8, device=DEV)
    want_s, bt_cpu, bt, status = summary.cpu().numpy(), bt.numpy(), bt.to(DEV), i32(1)
    lens, new = i32(B), i32(B)

    def append(q, k, v, slots, pos, max_new, qr):
        saw.saw_norm_rope_append(q, k, v, wq, wk, pos, cs, slots, qr, kc, vc, pages, P, True, True, h, dev_status=status)
        saw.saw_page_summary(kc, bt, lens, new, max_new, hkv, D, pages, P, summary, dev_status=status)

    lens.copy_(torch.tensor(prompts))
    new.copy_(lens)
    q, k, v = qkv(sum(prompts))
    slots = torch.cat([s[:n] for s, n in zip(slot_of, prompts)]).to(DEV)
    pos = torch.cat([torch.arange(n) for n in prompts]).int().to(DEV)
    append(q, k, v, slots, pos, max(prompts), torch.empty_like(q))
    torch.cuda.synchronize()
    summaries(want_s, kc.cpu().numpy(), bt_cpu, prompts, prompts, hkv, D, P, False)
    assert status.item() == 0
    assert_bytes_equal(summary, want_s, "summaries of the prompts")

    q, k, v = qkv(B)
    slots, pos, qr = i32(B), i32(B), torch.empty_like(q)
    out = torch.empty(B, hq, D, dtype=odt, device=DEV)
    tables, page_nos, sel_lens = i32(B, hkv, take), i32(B, hkv, take), i32(B, hkv)
    need = saw.saw_sparse_decode_workspace_bytes(B, hq, hkv, D, P, take * P)
    assert need > 0                                      # (the lists are split)
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)
    max_len = max(blocks) * P

    def step():
        append(q, k, v, slots, pos, 1, qr)
        saw.saw_select_pages(qr, summary, bt, lens, max_len, hkv, pages, P, True, h, first, last, tables, sel_lens,
                             sel_pages=page_nos, dev_status=status)
        saw.saw_sparse_decode_int4(qr, kc, vc, tables, sel_lens, take * P, hkv, pages, P, True, True, h, out, ws,
                                   dev_status=status)

    def prepare(n):
        for dst, src in zip((q, k, v), qkv(B)):
            dst.copy_(src)
        lens.copy_(torch.tensor([x + n for x in prompts]))
        new.fill_(1)
        pos.copy_(lens - 1)
        slots.copy_(torch.tensor([int(slot_of[b][x + n - 1]) for b, x in enumerate(prompts)]))

    def check(n):
        torch.cuda.synchronize()
        assert status.item() == 0
        now = [x + n for x in prompts]
        k_host, v_host, q_host = kc.cpu().numpy(), vc.cpu().numpy(), qr.float().cpu().numpy()
        summaries(want_s, k_host, bt_cpu, now, [1] * B, hkv, D, P, False)
        assert_bytes_equal(summary, want_s, "summaries")
        want = select(q_host, want_s, bt_cpu, now, hkv, D, P, True, h, take, first, last, False)
        for got, w in zip((tables, page_nos, sel_lens), want):
            assert np.array_equal(got.cpu().numpy(), w)
        ref, top, sd = attend(q_host, k_host, v_host, want[0], want[2], hkv, D, P, True, True, h, D ** -0.5, False, pages)
        # (the sparse decode's bound, with gains of up to 1.6 on either side of the logits)
        bound = 3 * 2.0 ** -14 * top + np.zeros_like(ref)
        if odt != torch.float32:
            bound += np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -7) + 5 * sd[..., None]
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()

    prepare(1)
    step()
    check(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(2, steps + 1):
        prepare(n)
        graph.replay()
        check(n)
