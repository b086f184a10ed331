"""Refusals of the serving-step entry points (tables, rotary append,
shared-prefix decode), on the CPU: every call carries one invalid argument
that the host checks catch, so nothing is launched on the made-up pointers."""
import pytest
import torch

import bit_paged_kv_gb300 as saw
from bit_paged_kv_gb300 import build as saw_build

A, B, C_, MIS = 0x10000, 0x20000, 0x30000, 0x10008
INV, UNS = saw.SAW_ERR_INVALID_ARG, saw.SAW_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    saw_build.build()
    return saw.lib()


def _tables(L, **kw):
    a = dict(src=A, rows=8, sblocks=4, srows=B, cached=A, new=B, free=A, nfree=16, count=None, B=4,
             T=8, pages=32, P=16, bt=B, mb=4, lens=C_, cu=A, slots=B, pos=A, taken=B, status=None)
    a.update(kw)
    return L.saw_build_tables(a["src"], a["rows"], a["sblocks"], a["srows"], a["cached"], a["new"],
                              a["free"], a["nfree"], a["count"], a["B"], a["T"], a["pages"], a["P"],
                              a["bt"], a["mb"], a["lens"], a["cu"], a["slots"], a["pos"], a["taken"],
                              a["status"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INV), (dict(T=-1), INV), (dict(pages=-1), INV), (dict(nfree=-1), INV),
    (dict(mb=-1), INV), (dict(rows=-1), INV), (dict(sblocks=-1), INV),
    (dict(P=8), UNS), (dict(B=65536), UNS), (dict(pages=1 << 28), UNS), (dict(mb=1 << 28), UNS),
    (dict(cu=None), INV), (dict(slots=None), INV), (dict(free=None), INV), (dict(new=None), INV),
    (dict(lens=None), INV), (dict(bt=None), INV),
    (dict(lens=A), INV),                          # seq_lens is cached_lens
    (dict(lens=B), INV),                          # seq_lens is new_lens
    (dict(src=B), INV),                           # in place with gathered rows
    (dict(src=B, srows=None, sblocks=5), INV),    # in place, another row length
    (dict(src=B, srows=None, rows=3), INV),       # in place, too few rows
])
def test_tables_refused(L, kw, expect):
    assert _tables(L, **kw) == expect


def _rope_table(L, **kw):
    a = dict(cs=A, n=64, r=64, base=1e4, kind=saw.SAW_ROPE_NONE, f=1.0, orig=0, low=0.0, high=0.0, att=0.0)
    a.update(kw)
    return L.saw_rope_table(a["cs"], a["n"], a["r"], a["base"], a["kind"], a["f"], a["orig"], a["low"],
                            a["high"], a["att"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(n=-1), INV), (dict(r=0), INV), (dict(r=24), UNS), (dict(r=272), UNS), (dict(base=1.0), INV),
    (dict(base=float("inf")), INV), (dict(base=float("nan")), INV), (dict(f=0.0), INV),
    (dict(f=float("nan")), INV), (dict(kind=5), INV), (dict(kind=-1), INV), (dict(att=-1.0), INV),
    (dict(kind=saw.SAW_ROPE_YARN), INV), (dict(kind=saw.SAW_ROPE_BANDS, orig=-1), INV),
    (dict(kind=saw.SAW_ROPE_BANDS, orig=64, low=4.0, high=1.0), INV),
    (dict(kind=saw.SAW_ROPE_YARN, orig=64, low=0.0, high=1.0), INV),
    (dict(kind=saw.SAW_ROPE_LINEAR, f=1e-320), INV),  # 1 / factor is infinite
    (dict(cs=None), INV), (dict(cs=MIS), INV), (dict(n=0), saw.SAW_OK),
])
def test_rope_table_refused(L, kw, expect):
    assert _rope_table(L, **kw) == expect


def _rope(L, **kw):
    a = dict(q=A, qs=4096, k=B, ks=1024, v=C_, vs=1024, pos=A, cs=B, n=64, r=128, inter=0, slots=A, T=4,
             hq=32, hkv=8, d=128, qo=A, qos=4096, kc=A, vc=B, pages=4, P=16, rk=1, rv=1, h=128, fmt=0)
    a.update(kw)
    return L.saw_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["cs"], a["n"],
                             a["r"], a["inter"], a["slots"], a["T"], a["hq"], a["hkv"], a["d"], a["qo"],
                             a["qos"], a["kc"], a["vc"], a["pages"], a["P"], a["rk"], a["rv"], a["h"],
                             a["fmt"], None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(T=-1), INV), (dict(hkv=0), INV), (dict(hq=-1), INV), (dict(n=-1), INV), (dict(pages=-1), INV),
    (dict(fmt=4), INV), (dict(d=96), UNS), (dict(P=8), UNS), (dict(r=0), INV), (dict(r=144), INV),
    (dict(r=24), UNS), (dict(inter=2), INV), (dict(rk=2), INV), (dict(rv=-1), INV), (dict(h=48), INV),
    (dict(h=256), INV), (dict(h=8), UNS), (dict(k=None), INV), (dict(pos=None), INV), (dict(cs=None), INV),
    (dict(slots=None), INV), (dict(kc=None), INV), (dict(vc=None), INV), (dict(qo=None), INV),
    (dict(q=MIS, qo=MIS), INV), (dict(k=MIS), INV), (dict(v=MIS), INV), (dict(kc=MIS), INV),
    (dict(cs=MIS), INV), (dict(qo=MIS), INV), (dict(ks=1020), INV), (dict(vs=1000), INV),
    (dict(qs=4092), INV), (dict(qos=4000, qo=B), INV),
    (dict(qs=8192), INV),                          # in place with another stride
    (dict(T=1 << 28), UNS), (dict(T=0), saw.SAW_OK),
])
def test_rope_append_refused(L, kw, expect):
    assert _rope(L, **kw) == expect


def _prefix(L, **kw):
    a = dict(q=A, kc=A, vc=B, bt=A, mb=8, sl=B, cu=A, pre=B, groups=1, B=2, maxp=64, maxo=64, hq=32, hkv=8,
             d=128, pages=8, P=16, rk=1, rv=1, h=128, scale=0.0, out=A, ws=B, wsb=1 << 40, mode=0, fmt=4)
    a.update(kw)
    return L.saw_prefix_decode_int4(a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["sl"], a["cu"], a["pre"],
                                    a["groups"], a["B"], a["maxp"], a["maxo"], a["hq"], a["hkv"], a["d"],
                                    a["pages"], a["P"], a["rk"], a["rv"], a["h"], a["scale"], a["out"],
                                    a["ws"], a["wsb"], a["mode"], a["fmt"], None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(d=64), UNS), (dict(P=8), UNS), (dict(hq=12), INV), (dict(hq=72), UNS), (dict(B=-1), INV),
    (dict(groups=-1), INV), (dict(maxp=-1), INV), (dict(maxo=-1), INV), (dict(maxp=1 << 30, maxo=1 << 30), INV),
    (dict(maxp=129), INV),                         # beyond the tables
    (dict(mb=-1), INV), (dict(cu=None), INV), (dict(pre=None), INV), (dict(q=None), INV), (dict(kc=None), INV),
    (dict(bt=None), INV), (dict(sl=None), INV), (dict(out=None), INV), (dict(out=MIS), INV), (dict(q=MIS), INV),
    (dict(scale=-1.0), INV), (dict(scale=float("nan")), INV), (dict(fmt=8), INV), (dict(h=48), INV),
    (dict(rk=2), INV), (dict(hkv=0), INV), (dict(mode=3), INV), (dict(mode=-1), INV), (dict(groups=65536), UNS),
    (dict(B=0), saw.SAW_OK),
])
def test_prefix_refused(L, kw, expect):
    assert _prefix(L, **kw) == expect


def test_prefix_workspace_refused(L):
    args = (64, 1, 32, 8, 128, 16, 16384, 2048)
    need = saw.saw_prefix_decode_workspace_bytes(*args)
    assert need > 0
    big = dict(B=64, maxp=16384, maxo=2048, mb=2048, pages=4096)
    assert _prefix(L, **big, ws=None) == INV
    assert _prefix(L, **big, ws=MIS) == INV
    assert _prefix(L, **big, wsb=need - 1) == INV
    # small sizes read every table apart: no more than the decode's own workspace
    small = (4, 1, 32, 8, 128, 16, 64, 64)
    assert saw.saw_prefix_decode_workspace_bytes(*small) == 0
    assert saw.saw_prefix_decode_workspace_bytes(*small, saw.SAW_PREFIX_SHARE) > 0
    assert saw.saw_prefix_decode_workspace_bytes(*small, 7) == 0
    assert _prefix(L, mode=saw.SAW_PREFIX_SHARE, wsb=1 << 20) == INV
    assert saw.saw_prefix_decode_workspace_bytes(64, 1, 32, 8, 64, 16, 16384, 2048) == 0
    assert saw.saw_prefix_decode_workspace_bytes(-1, 1, 32, 8, 128, 16, 16384, 2048) == 0


def test_status_name():
    assert saw.saw_status_string(saw.SAW_ERR_DEVICE_PAGES) == "SAW_ERR_DEVICE_PAGES"


def test_binding_refuses_other_devices():
    """Tensors that are not on the current CUDA device are refused in Python."""
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        saw.saw_build_tables(t, t, t, None, 16, 8, t.view(4, 1), t, t, t)
