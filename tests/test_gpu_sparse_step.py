"""A sparse decode step as a server runs it: tables, the normed rotary append, the
summaries of completed pages, the selection and the decode over its lists, from
prompts on, eager and as one replayed graph.  The caches, summaries and lists are
checked byte for byte, the attention in 64 bits over the lists."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from gpu_helpers import assert_bytes_equal
from sparse_oracle import attend, norm_rows, select, summaries
from test_gpu_rope import oracle_cache, turn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(*s):
    return torch.zeros(s, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("D,hq,hkv,P,prompts,take", [(128, 8, 2, 16, [900, 95, 16, 1], 9), (64, 4, 4, 32, [700, 31], 5),
                                                     (256, 16, 2, 16, [400, 333, 47], 12)])
def test_prompts_and_decode_steps(D, hq, hkv, P, prompts, take):
    B, steps, first, last, h, eps = len(prompts), 6, 1, 2, 64, 1e-6
    T = sum(prompts)
    blocks = -(-(max(prompts) + steps) // P)
    pages = sum(-(-(n + steps) // P) for n in prompts) + 3
    g = torch.Generator(device=DEV).manual_seed(D)
    qkv = lambda n: [torch.randn(n, x, D, generator=g, device=DEV).bfloat16() for x in (hq, hkv, hkv)]
    wq, wk = (1 + 0.2 * torch.randn(2, D, generator=g, device=DEV)).bfloat16()
    cs = torch.empty(2048, D, device=DEV)
    saw.saw_rope_table(cs, 1e6)
    n = saw.saw_cache_bytes(pages, P, hkv, D)
    kc, vc = (torch.full((n,), 0xAB, dtype=torch.uint8, device=DEV) for _ in range(2))
    summary = torch.full((saw.saw_summary_bytes(pages, hkv, D),), 0xAB, dtype=torch.uint8, device=DEV)
    free = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).int().to(DEV)
    status = i32(1)
    bt, lens, cu, taken = i32(B, blocks) - 1, i32(B), i32(B + 1), i32(1)
    want_k, want_v, want_s = kc.cpu().numpy(), vc.cpu().numpy(), summary.cpu().numpy()

    def append(q, k, v, cached, new, max_new, slots, pos, qr, free):
        saw.saw_build_tables(cached, new, free, None, P, pages, bt, lens, cu, slots, pos, taken,
                             src_tables=None if cached is None else bt, dev_status=status)
        saw.saw_norm_rope_append(q, k, v, wq, wk, pos, cs, slots, qr, kc, vc, pages, P, True, True, h, eps=eps,
                                 dev_status=status)
        saw.saw_page_summary(kc, bt, lens, new, max_new, hkv, D, pages, P, summary, dev_status=status)

    def check_append(q, k, v, new, slots, pos, qr):
        f32 = lambda x: x.float().cpu().numpy()
        rows, sl = cs[pos.long()].cpu().numpy(), slots.cpu().numpy()
        for cache, want, x in ((kc, want_k, turn(norm_rows(f32(k), f32(wk), 0.0, eps), rows, D, False)), (vc, want_v, f32(v))):
            fresh = oracle_cache(x, sl, pages, P, True, h, False)
            # (oracle_cache starts from 0xAB everywhere: take the rows written)
            at = oracle_cache(np.zeros_like(x), sl, pages, P, True, h, False)
            rows_set = at != 0xAB
            want[rows_set] = fresh[rows_set]
            assert_bytes_equal(cache, want, "cache")
        y = turn(norm_rows(f32(q), f32(wq), 0.0, eps), rows, D, False)
        assert torch.equal(qr, torch.from_numpy(y).bfloat16().to(DEV))
        summaries(want_s, want_k, bt.cpu().numpy(), lens.tolist(), new.tolist(), hkv, D, P, False)
        assert_bytes_equal(summary, want_s, "summaries")

    q, k, v = qkv(T)
    new = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    slots, pos, qr = i32(T), i32(T), torch.empty_like(q)
    append(q, k, v, None, new, max(prompts), slots, pos, qr, free)
    torch.cuda.synchronize()
    assert status.item() == 0
    check_append(q, k, v, new, slots, pos, qr)
    free = free[int(taken.item()):].contiguous()

    cached, one, slots, pos = lens.clone(), i32(B) + 1, i32(B), i32(B)
    q, k, v = qkv(B)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    max_len = blocks * P
    tables, page_nos, sel_lens = i32(B, hkv, take), i32(B, hkv, take), i32(B, hkv)
    need = saw.saw_sparse_decode_workspace_bytes(B, hq, hkv, D, P, take * P)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    used = i32(1)

    def step():
        append(q, k, v, cached, one, 1, slots, pos, qr, free)
        saw.saw_select_pages(qr, summary, bt, lens, max_len, hkv, pages, P, True, h, first, last, tables, sel_lens,
                             sel_pages=page_nos, dev_status=status)
        saw.saw_sparse_decode_int4(qr, kc, vc, tables, sel_lens, take * P, hkv, pages, P, True, True, h, out, ws,
                                   dev_status=status)
        cached.copy_(lens)
        # the pages taken leave the list
        used.copy_(taken)
        at = (torch.arange(free.numel(), device=DEV) + used) % free.numel()
        free.copy_(free[at])

    def check(n):
        torch.cuda.synchronize()
        assert status.item() == 0
        assert lens.tolist() == [x + n for x in prompts]
        check_append(q, k, v, one, slots, pos, qr)
        want = select(qr.float().cpu().numpy(), want_s, bt.cpu().numpy(), lens.tolist(), hkv, D, P, True, h, take, first,
                      last, False)
        for got, w in zip((tables, page_nos, sel_lens), want):
            assert np.array_equal(got.cpu().numpy(), w)
        ref, top, sd = attend(qr.float().cpu().numpy(), want_k, want_v, want[0], want[2], hkv, D, P, True, True, h,
                              D ** -0.5, False, pages)
        # (the bound of the sparse decode's own tests; gains of up to 1.6 on either side of the logits)
        bound = 3 * 2.0 ** -14 * top + np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -7) + 5 * sd[..., None]
        assert (np.abs(out.double().cpu().numpy() - ref) <= bound).all()

    for n in range(1, 3):
        for dst, src in zip((q, k, v), qkv(B)):
            dst.copy_(src)
        step()
        check(n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(3, steps + 1):
        for dst, src in zip((q, k, v), qkv(B)):
            dst.copy_(src)
        graph.replay()
        check(n)
