"""saw_build_tables as a server calls it: from several threads at once, and in
place in tables with more rows than the batch."""
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from conftest import ROOT
from test_gpu_tables import batch, check, model

pytestmark = pytest.mark.gpu


def test_threads_at_once():
    """Eight threads, batches of two sizes that want more than 48 KB of shared memory: every call is launched, every
    batch right."""
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    L, sides = saw.lib(), []
    for B in (2500, 4096) * 4:
        cached, fresh, free, pages, blocks, src, rows = batch(B, B, 60, 2, 16)
        T = int(fresh.sum())
        bt = np.full((B, blocks), -7, np.int32)
        want, _ = model(cached, fresh, free, len(free), 16, pages, blocks, T, src, rows, bt)
        out = dict(bt=i32(bt), lens=i32(np.zeros(B)), cu=i32(np.zeros(B + 1)), slots=i32(np.zeros(T)),
                   pos=i32(np.zeros(T)), taken=i32([0]))
        ins = [i32(x) for x in (src, rows, cached, fresh, free)]
        stream = torch.cuda.Stream()
        s, r, c, n, f = (x.data_ptr() for x in ins)
        o = {k: v.data_ptr() for k, v in out.items()}
        args = (s, len(src), blocks, r, c, n, f, len(free), None, B, T, pages, 16, o["bt"], blocks, o["lens"], o["cu"],
                o["slots"], o["pos"], o["taken"], None, stream.cuda_stream)
        sides.append((args, want, out, stream, ins))
    torch.cuda.synchronize()
    failed = []

    def work(args):
        with torch.cuda.device(0):
            failed.append(sum(L.saw_build_tables(*args) != saw.SAW_OK for _ in range(5000)))

    threads = [threading.Thread(target=work, args=(side[0],)) for side in sides]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert failed == [0] * 8
    for _, want, out, *_ in sides:
        assert all(np.array_equal(out[k].cpu().numpy(), want[k]) for k in want)


SIZES = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import bit_paged_kv_gb300 as saw
i32 = lambda n, v=0: torch.full((n,), v, dtype=torch.int32, device="cuda")
for B in range(2370, 2420):
    lens, cu, slots, taken = i32(B), i32(B + 1), i32(B), i32(1)
    saw.saw_build_tables(None, i32(B, 1), torch.arange(B, device="cuda", dtype=torch.int32), None, 16, B,
                         i32(B).view(B, 1), lens, cu, slots, pages_taken=taken)
    assert taken.item() == B and lens.sum().item() == B and (slots == 16 * torch.arange(B, device="cuda")).all(), B
"""


def test_every_size_around_the_shared_memory_limit():
    """Batches whose sums take just under and over 48 KB, in a process that launched no larger one before."""
    r = subprocess.run([sys.executable, "-c", SIZES, ROOT], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("B,more", [(1, 1), (5, 3), (70, 1), (200, 130), (4500, 60)])
def test_in_place_leaves_the_rows_behind_the_batch(B, more):
    """A server's table of more rows than the batch, every row with pages, extended in place: the batch's rows get
    their new entries, the rows behind it keep all of theirs."""
    cached, fresh, free, pages, blocks, src, rows = batch(B, B, 300, 20, 16, extra_rows=0)
    src = np.concatenate((src[rows], np.random.default_rng(1).integers(0, pages, (more, blocks)))).astype(np.int32)
    T = int(fresh.sum()) + 3
    want, codes = model(cached, fresh, free, len(free), 16, pages, blocks, T, src, None, src[:B])
    whole = torch.from_numpy(src).cuda()
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    out = dict(bt=whole[:B], lens=i32(np.zeros(B)), cu=i32(np.zeros(B + 1)), slots=i32(np.zeros(T)),
               pos=i32(np.zeros(T)), taken=i32([0]))
    status = i32([0])
    saw.saw_build_tables(i32(cached), i32(fresh), i32(free), None, 16, pages, *out.values(), whole, None, status)
    assert status.item() == 0 and not codes
    for k in want:
        assert np.array_equal(out[k].cpu().numpy(), want[k]), k
    assert np.array_equal(whole[B:].cpu().numpy(), src[B:])


@pytest.mark.parametrize("B", [4096, 4097, 8191, 11263, 11264, 11265, 65535])
@pytest.mark.parametrize("lists", ["all", "half"])
def test_large_batches(B, lists):
    """Around the largest batch whose sums fit shared memory one by one, and the largest of all; the free list covers
    all of it, or half."""
    check(*batch_args(B, lists))


def batch_args(B, lists):
    cached, fresh, free, pages, blocks, src, rows = batch(B, B, 40, 3, 16)
    nfree = len(free) if lists == "all" else len(free) // 2
    return cached, fresh, free, nfree, 16, pages, blocks, int(fresh.sum()) + 2, src, rows
