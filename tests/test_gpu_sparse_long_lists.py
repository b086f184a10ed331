"""saw_sparse_decode_int4 over lists that are longer than what a warp holds of their
page ids: 64 steps at head_dim 256, 256 at smaller ones, beyond which the ids are
read as the pages are.  Lists this long among as many units as leave them unsplit."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from test_gpu_sparse_decode import check, make

pytestmark = pytest.mark.gpu


def long_case(D, hq, P, n, units, seed):
    """units lists of which the first has n tokens, one 333, the others none; few pages, listed over and over."""
    rng = np.random.default_rng(seed)
    B, hkv = units // 2, 2
    q, kc, vc, _, _, pages = make(seed, [[90 * P, 80 * P]], hq, hkv, D, P, torch.float16, False)
    q = torch.randn(B, hq, D, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").half()
    lens = np.zeros((B, hkv), np.int32)
    lens[0, 0], lens[B - 1, 1] = n, 333
    tables = np.full((B, hkv, -(-n // P)), -1, np.int32)
    tables[0, 0] = rng.integers(0, pages, tables.shape[-1])
    tables[B - 1, 1] = rng.integers(0, pages, tables.shape[-1])
    return q, kc, vc, tables, lens, pages


@pytest.mark.parametrize("units", [152, 432, 592])
@pytest.mark.parametrize("D,hq,P,n", [(256, 4, 16, 64 * 16 * 16 + 100), (256, 12, 64, 64 * 16 * 16 + 33),
                                      (128, 8, 16, 256 * 4 * 16 + 7), (64, 12, 32, 256 * 4 * 16 + 500)])
def test_beyond_the_held_ids(D, hq, P, n, units):
    """The largest CTA at head_dim 256, 4-warp CTAs' worth at smaller ones; grids that take 16 warps and fewer."""
    check(*long_case(D, hq, P, n, units, D + units), P, True, True, 64, False)


@pytest.mark.parametrize("D,hq,P,n", [(128, 8, 32, 256 * 16 * 16 + 40), (256, 2, 16, 64 * 16 * 16 + 300)])
def test_bad_pages_beyond_the_held_ids(D, hq, P, n):
    q, kc, vc, tables, lens, pages = long_case(D, hq, P, n, 152, 5)
    check(q, kc, vc, tables, lens, pages, P, True, True, 64, False)
    t = tables.copy()
    t[0, 0, [-2, -3, 7]] = -1, pages, 2 ** 31 - 1
    check(q, kc, vc, t, lens, pages, P, True, True, 64, False, status=saw.SAW_ERR_DEVICE_INDEX)
