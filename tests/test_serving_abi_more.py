"""Limits of the serving-step entry points, on the CPU: one argument beyond
each, on made-up pointers that nothing is launched on."""
import pytest

import bit_paged_kv_gb300 as saw
from test_serving_abi import INV, L, UNS, _rope  # noqa: F401


@pytest.mark.parametrize("kw,expect", [
    (dict(T=1, hq=65536, qs=1 << 23, qos=1 << 23), UNS), (dict(T=1, hq=1 << 24, qs=1 << 31, qos=1 << 31), UNS),
    (dict(T=1, hkv=65536, ks=1 << 23, vs=1 << 23), UNS), (dict(T=1, hkv=1 << 29, ks=1 << 36, vs=1 << 36), UNS),
    (dict(T=(1 << 30) // 48, hq=32, hkv=8, pos=None), INV),  # within: the next check speaks
    (dict(T=(1 << 30) // 48 + 1, hq=32, hkv=8, pos=None), UNS),
    (dict(T=1, hq=65535, qs=1 << 23, qos=1 << 23, pos=None), INV),
])
def test_rope_append_limits(L, kw, expect):  # noqa: F811
    assert _rope(L, **kw) == expect
