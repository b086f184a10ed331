"""Refusals of the sparse decode step's entry points, on the CPU: every call
carries one invalid argument that the host checks catch, so nothing is launched
on the made-up pointers."""
import math

import pytest

import bit_paged_kv_gb300 as saw
from bit_paged_kv_gb300 import build as saw_build

A, B, C_, MIS = 0x10000, 0x20000, 0x30000, 0x10008
INV, UNS, OK = saw.SAW_ERR_INVALID_ARG, saw.SAW_ERR_UNSUPPORTED, saw.SAW_OK
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def L():
    saw_build.build()
    return saw.lib()


def _norm(L, **kw):
    a = dict(q=A, qs=4096, k=B, ks=1024, v=C_, vs=1024, wq=A, wk=B, off=0.0, eps=1e-6, pos=A, cs=B, n=64, r=128,
             inter=0, slots=A, T=4, hq=32, hkv=8, d=128, qo=A, qos=4096, kc=A, vc=B, pages=4, P=16, rk=1, rv=1, h=128,
             fmt=0)
    a.update(kw)
    return L.saw_norm_rope_append(*a.values(), None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(eps=0.0), INV), (dict(eps=-1e-6), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(eps=1e-31), INV), (dict(off=NAN), INV),
    (dict(off=INF), INV), (dict(wq=MIS), INV), (dict(wk=MIS), INV), (dict(fmt=4), INV), (dict(fmt=16), INV),
    (dict(fmt=12), INV), (dict(T=-1), INV), (dict(hkv=0), INV), (dict(d=96), UNS), (dict(P=8), UNS), (dict(r=24), UNS),
    (dict(inter=2), INV), (dict(h=48), INV), (dict(k=None), INV), (dict(qo=None), INV), (dict(vc=None), INV),
    (dict(q=MIS, qo=MIS), INV), (dict(qs=8192), INV), (dict(ks=1020), INV), (dict(T=1 << 28), UNS), (dict(T=0), OK),
    (dict(T=0, wq=None, wk=None, fmt=11), OK), (dict(T=0, eps=0.0), INV),
])
def test_norm_rope_append_refused(L, kw, expect):
    assert _norm(L, **kw) == expect


def test_summary_bytes():
    assert saw.saw_summary_bytes(1, 8, 128) == 8 * 68
    assert saw.saw_summary_bytes(10, 3, 64) == 10 * 112  # 3 * 36 up to a multiple of 16
    assert saw.saw_summary_bytes(1 << 20, 8, 256) == (1 << 20) * 1056
    for bad in ((0, 8, 128), (-1, 8, 128), (4, 0, 128), (4, 8, 0), (4, 8, -128), (4, 8, 127)):
        assert saw.saw_summary_bytes(*bad) == 0


def _summary(L, **kw):
    a = dict(kc=A, bt=B, mb=8, lens=A, new=B, B=2, maxn=16, hkv=8, d=128, pages=8, P=16, out=C_, fmt=0)
    a.update(kw)
    return L.saw_page_summary(*a.values(), None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INV), (dict(hkv=0), INV), (dict(pages=-1), INV), (dict(mb=-1), INV), (dict(maxn=-1), INV),
    (dict(fmt=1), INV), (dict(fmt=4), INV), (dict(d=96), UNS), (dict(P=8), UNS), (dict(B=65536), UNS),
    (dict(hkv=65536), UNS), (dict(maxn=2 ** 31 - 1, hkv=9), UNS), (dict(kc=None), INV), (dict(bt=None), INV),
    (dict(lens=None), INV), (dict(out=None), INV), (dict(kc=MIS), INV), (dict(out=MIS), INV), (dict(B=0), OK),
])
def test_page_summary_refused(L, kw, expect):
    assert _summary(L, **kw) == expect


def _select(L, **kw):
    a = dict(q=A, s=B, bt=A, mb=64, lens=B, B=2, maxl=1024, hq=32, hkv=8, d=128, pages=8, P=16, rk=1, h=128, take=8,
             first=1, last=2, tab=C_, pg=C_, sl=C_, fmt=0)
    a.update(kw)
    return L.saw_select_pages(*a.values(), None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INV), (dict(hkv=0), INV), (dict(hq=0), INV), (dict(hq=12), INV), (dict(hq=72), UNS), (dict(pages=-1), INV),
    (dict(maxl=-1), INV), (dict(mb=-1), INV), (dict(mb=63), INV), (dict(fmt=4), INV), (dict(fmt=8), INV),
    (dict(d=96), UNS), (dict(P=8), UNS), (dict(rk=2), INV), (dict(h=48), INV), (dict(h=256), INV), (dict(h=8), UNS),
    (dict(take=0), INV), (dict(take=2), INV), (dict(first=-1), INV), (dict(last=0), INV),
    (dict(first=2 ** 31 - 1), INV), (dict(take=(1 << 18) + 1), UNS), (dict(maxl=(1 << 22) + 1, mb=(1 << 18) + 1), UNS),
    (dict(B=65536), UNS), (dict(hkv=65536, hq=65536), UNS), (dict(q=None), INV), (dict(s=None), INV), (dict(bt=None), INV),
    (dict(lens=None), INV), (dict(tab=None), INV), (dict(sl=None), INV), (dict(q=MIS), INV), (dict(s=MIS), INV),
    (dict(B=0), OK), (dict(B=0, rk=0, h=48), OK),
])
def test_select_pages_refused(L, kw, expect):
    assert _select(L, **kw) == expect


def _sparse(L, **kw):
    a = dict(q=A, kc=A, vc=B, tab=A, sel=128, lens=B, B=2, maxl=1024, hq=32, hkv=8, d=128, pages=8, P=16, rk=1, rv=1,
             h=128, scale=0.0, out=C_, ws=C_, wsb=1 << 40, fmt=0)
    a.update(kw)
    return L.saw_sparse_decode_int4(*a.values(), None, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=-1), INV), (dict(sel=-1), INV), (dict(sel=63), INV), (dict(maxl=-1), INV), (dict(hq=12), INV),
    (dict(hq=72), UNS), (dict(hkv=0), INV), (dict(d=96), UNS), (dict(P=8), UNS), (dict(fmt=8), INV), (dict(rk=2), INV),
    (dict(rv=2), INV), (dict(h=48), INV), (dict(h=8), UNS), (dict(scale=-1.0), INV), (dict(scale=NAN), INV),
    (dict(scale=INF), INV), (dict(q=None), INV), (dict(kc=None), INV), (dict(vc=None), INV), (dict(tab=None), INV),
    (dict(lens=None), INV), (dict(out=None), INV), (dict(q=MIS), INV), (dict(out=MIS), INV), (dict(kc=MIS), INV),
    (dict(B=65536), UNS), (dict(B=0), OK), (dict(B=0, fmt=7), OK),
])
def test_sparse_decode_refused(L, kw, expect):
    assert _sparse(L, **kw) == expect


def test_sparse_workspace(L):
    args = (1, 32, 8, 128, 16, 65536)
    need = saw.saw_sparse_decode_workspace_bytes(*args)
    assert need > 1 << 20
    big = dict(B=1, maxl=65536, sel=4096)
    assert _sparse(L, **big, ws=None) == INV
    assert _sparse(L, **big, ws=MIS) == INV
    assert _sparse(L, **big, wsb=need - 1) == INV
    assert saw.saw_sparse_decode_workspace_bytes(512, 32, 8, 128, 16, 256) == 0
    for bad in ((-1, 32, 8, 128, 16, 65536), (1, 0, 8, 128, 16, 65536), (1, 32, 0, 128, 16, 65536),
                (1, 32, 8, 96, 16, 65536), (1, 32, 8, 128, 8, 65536), (1, 32, 8, 128, 16, -1)):
        assert saw.saw_sparse_decode_workspace_bytes(*bad) == 0
