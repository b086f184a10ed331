"""The serving-step operators together, as a server runs them: tables, rotary
append of a shared prompt, forked requests, then decode steps of tables,
rotary append and shared-prefix attention, eager and as one replayed graph.
The reference keeps every token's q, k and v, turns them and attends in
float64 over the rows as the caches hold them.

Bar of the attention: 2e-3 of the largest output, or ABS where that is more.
These rows are pure noise, so a softmax over n of them leaves outputs of about
n^-1/2, while the decode's binary16 rounding of p s_V does not shrink with
them: token j's rounding d_j (uniform within 2^-11 of p_j s_j at most, so of
standard deviation 2^-11 / sqrt(3) of it at most) multiplies codes whose mean
over the 128 rotated dims is 7.5, and the inverse rotation gathers that common
part into one dim as 7.5 sqrt(128) d_j.  With s <= 0.4 (128 normal values span
at most 6), unit-variance logits (sqrt(sum p^2) = sqrt(e / n), n >= 480) and
independent roundings, one standard deviation is
7.5 * 11.3 * 0.4 * 2^-11 / sqrt(3) * 0.0753 = 7.2e-4; ABS is three of them.
"""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
import oracle
from gpu_helpers import ATTN_TOL, bits, rel_err

pytestmark = pytest.mark.gpu
DEV = "cuda"
ABS = 3 * 7.2e-4


class Server:
    """Buffers of a small server: B requests behind one prompt."""

    def __init__(self, B, P, hq, hkv, pages, blocks):
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
        self.B, self.P, self.hq, self.hkv, self.pages, self.blocks = B, P, hq, hkv, pages, blocks
        n = saw.saw_cache_bytes(pages, P, hkv, 128)
        self.kc = torch.zeros(n, dtype=torch.uint8, device=DEV)
        self.vc = torch.zeros(n, dtype=torch.uint8, device=DEV)
        self.cs = torch.empty(4096, 128, device=DEV)
        saw.saw_rope_table(self.cs, 1e6, saw.SAW_ROPE_YARN, 4.0, 1024)
        self.free = torch.randperm(pages, generator=torch.Generator().manual_seed(2)).int().to(DEV)
        self.status = z(1)
        self.bt, self.lens, self.cu = z(B, blocks), z(B), z(B + 1)

    def tables(self, cached, new, slots, pos, taken, bt, lens, cu, free, src=None, rows=None):
        saw.saw_build_tables(cached, new, free, None, self.P, self.pages, bt, lens, cu, slots, pos, taken,
                             src_tables=src, src_rows=rows, dev_status=self.status)

    def append(self, q, k, v, pos, slots, q_out):
        saw.saw_rope_append(q, k, v, pos, self.cs, slots, q_out, self.kc, self.vc, self.pages, self.P, True, True, 128,
                            dev_status=self.status)


def test_prompt_fork_and_decode_steps():
    B, P, hq, hkv, prompt, steps = 40, 16, 16, 4, 16 * 30, 5
    sv = Server(B, P, hq, hkv, 30 + B * 2 + 4, 36)
    g = torch.Generator(device=DEV).manual_seed(0)
    qkv = lambda n: [torch.randn(n, h, 128, generator=g, device=DEV).bfloat16() for h in (hq, hkv, hkv)]
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    # the prompt, once: request row 0
    q, k, v = qkv(prompt)
    bt0, lens0, cu0, slots, pos, taken = i32(1, sv.blocks) - 1, i32(1), i32(2), i32(prompt), i32(prompt), i32(1)
    sv.tables(None, torch.tensor([prompt], dtype=torch.int32, device=DEV), slots, pos, taken, bt0, lens0, cu0, sv.free)
    qr = torch.empty_like(q)
    sv.append(q, k, v, pos, slots, qr)
    out0 = torch.empty(prompt, hq, 128, device=DEV)
    saw.saw_prefill_attn_int4(qr, cu0, sv.kc, sv.vc, bt0, lens0, prompt, prompt, hkv, sv.pages, P, True, True, 128, out0,
                              dev_status=sv.status)
    torch.cuda.synchronize()
    assert sv.status.item() == 0 and taken.item() == 30
    # every request forks it and decodes step by step
    free = sv.free[30:].contiguous()
    cached = i32(B) + prompt
    one, fork = i32(B) + 1, i32(B)
    cu_g, pre = torch.tensor([0, B], dtype=torch.int32, device=DEV), torch.tensor([prompt], dtype=torch.int32, device=DEV)
    max_own = 64
    need = saw.saw_prefix_decode_workspace_bytes(B, 1, hq, hkv, 128, P, prompt, max_own)
    ws = torch.zeros(max(need, 16), dtype=torch.uint8, device=DEV)
    slots, pos, qr, out = i32(B), i32(B), torch.empty(B, hq, 128, dtype=torch.bfloat16, device=DEV), torch.empty(B, hq, 128, device=DEV)
    bt, lens = i32(B, sv.blocks) - 1, i32(B)
    qi, ki, vi = [torch.zeros(B, h, 128, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv)]

    def step(first):
        sv.tables(cached, one, slots, pos, taken, bt, lens, sv.cu, free, bt0 if first else bt, fork if first else None)
        sv.append(qi, ki, vi, pos, slots, qr)
        saw.saw_prefix_decode_int4(qr, sv.kc, sv.vc, bt, lens, cu_g, pre, prompt, max_own, hkv, sv.pages, P, True, True,
                                   128, out, ws, dev_status=sv.status)
        cached.copy_(lens)

    def check(n):
        torch.cuda.synchronize()
        assert sv.status.item() == 0
        assert (lens == prompt + n).all() and (pos == prompt + n - 1).all()
        ref = oracle.decode(bits(qr), sv.kc.cpu().numpy(), sv.vc.cpu().numpy(), bt.cpu().numpy(), lens.cpu().numpy(), hq,
                            hkv, 128, sv.pages, P, True, True, 128, threads=oracle.host_threads())
        err = rel_err(out.cpu().numpy().reshape(-1, 128), ref, "serving-step") * np.abs(ref).max()
        assert err <= max(ATTN_TOL * np.abs(ref).max(), ABS)
        # the step's q against the definition
        cs = sv.cs[pos.long()].double().cpu().numpy()[:, None]
        x = qi.double().cpu().numpy()
        c, s = cs[..., :64], cs[..., 64:]
        y = np.concatenate((x[..., :64] * c - x[..., 64:] * s, x[..., 64:] * c + x[..., :64] * s), -1)
        assert np.abs(qr.double().cpu().numpy() - y).max() <= (2.0 ** -9 + 2.0 ** -21) * np.abs(y).max() * 2

    for n in range(1, 3):
        for dst, src in zip((qi, ki, vi), qkv(B)):
            dst.copy_(src)
        step(n == 1)
        if n == 1:
            free = free[int(taken.item()):].contiguous()
        check(n)
    # the same step as one graph, replayed
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(False)
    for n in range(3, steps + 1):
        for dst, src in zip((qi, ki, vi), qkv(B)):
            dst.copy_(src)
        graph.replay()
        check(n)
