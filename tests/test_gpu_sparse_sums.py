"""saw_sparse_decode_int4's sums: p s carried to 22 bits (but for bfloat16 outputs of
more than 4 q-heads per kv-head), and products that are small beside others of their
tile.

Keys are constant rows of whole numbers and the softmax scale makes the base-2 score
half of them, exactly: a weight 2^(-c/2) is off by ex2's 2^-22.  The tensor cores add 16
products and the sum so far, each cut towards zero at 2^-25 of 2^E, E the largest of
their exponents, a subnormal operand's counting as -14 (measured): codes n 2^-21 beside
2^e <= p s < 2^(e + 1) are cut at 2^(e - 14 - 25), 2^-18 of a code step of the tile's
largest p s, 17 of them a tile, or at 2^-25 of the sum so far."""
import numpy as np
import pytest
import torch

import bit_paged_kv_gb300 as saw
from sparse_oracle import rows_of
from test_gpu_sparse_decode import run

pytestmark = pytest.mark.gpu
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SCALE = float(np.float32(0.5 / 1.4426950408889634))
HALF = float(np.float32(SCALE * 1.4426950408889634))    # of a score, as the library rounds it
assert HALF == 0.5
# of sum w (n s + |z|): the weights, twice 2^-22; one tile per warp, two products' sums cut at 17 2^-25;
# warps, the sum of the weights and the quotient in at most 34 roundings of 2^-24; p s 2^-22
RELATIVE = 2.0 ** -18


def case(seed, c, v, lens, hq, hkv, P, dt, meta):
    """Tokens in the order of the lists: keys -c [T], values v [T, hkv, D]."""
    T, _, D = v.shape
    pages = T // P
    n = saw.saw_cache_bytes(pages, P, hkv, D)
    kc, vc = (torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    k = torch.tensor(-c, dtype=dt).cuda()[:, None, None].expand(T, hkv, D).contiguous()
    saw.saw_quantize_append(k, torch.from_numpy(v.astype(np.float32)).to(dt).cuda(), torch.arange(T, device="cuda").int(),
                            kc, vc, pages, P, False, False, 64, meta_bf16=meta)
    B = len(lens)
    tables = np.broadcast_to(np.arange(pages, dtype=np.int32), (B, hkv, pages)).copy()
    q = torch.zeros(B, hq, D, dtype=dt, device="cuda")
    q[:, :, 0] = 1
    return q, kc, vc, tables, np.repeat(np.asarray(lens, np.int32)[:, None], hkv, 1), pages


def check(got_case, hkv, P, meta, odt):
    q, kc, vc, tables, lens, pages = got_case
    out, st = run(q, kc, vc, tables, lens, pages, P, False, False, 64, meta, odt=odt, scale=SCALE)
    assert st == 0
    G, D = q.shape[1] // hkv, q.shape[2]
    got, kn, vn = out.double().cpu().numpy(), kc.cpu().numpy(), vc.cpu().numpy()
    for h in range(hkv):
        rows = [[rows_of(x, e, h, hkv, D, P, meta) for e in range(pages)] for x in (kn, vn)]
        K = np.concatenate([r[2] for r in rows[0]]).astype(np.float64)
        c, s, z = (np.concatenate([r[i] for r in rows[1]]).astype(np.float64) for i in range(3))
        for b, n in enumerate(lens[:, h]):
            w = 2.0 ** (K[:n] * HALF)
            w /= w.sum()
            ref = w @ (c[:n] * s[:n, None] + z[:n, None])
            tiles = np.pad(w * s[:n], (0, -n % 16)).reshape(-1, 16).max(-1).sum()
            bound = RELATIVE * (w @ (c[:n] * s[:n, None] + np.abs(z[:n, None]))) + 17 * 2.0 ** -18 * tiles
            if out.dtype != F32:
                fi = torch.finfo(out.dtype)
                bound = bound + np.maximum(np.abs(ref) * (fi.eps / 2) * (1 + 2.0 ** -7), fi.tiny * fi.eps / 2)
            err = np.abs(got[b, h * G:(h + 1) * G] - ref)
            assert (err <= bound).all(), (b, h, float((err / bound).max()))


SHAPES = [(64, 3, 1, 16), (64, 8, 1, 32), (128, 8, 2, 16), (128, 1, 1, 64), (128, 16, 2, 16), (256, 4, 2, 32), (256, 6, 1, 16)]
OUTPUTS = [(BF, BF, False), (BF, F32, False), (F16, F16, True), (F16, F32, False)]


# (bfloat16 outputs of more than 4 q-heads per kv-head: 11 bits of p s)
CASES = [(*shape, *out) for shape in SHAPES for out in OUTPUTS if out[1] != BF or shape[1] <= 4 * shape[2]]


@pytest.mark.parametrize("D,hq,hkv,P,dt,odt,meta", CASES)
def test_weights_times_scales(D, hq, hkv, P, dt, odt, meta):
    """Few tokens, up to 9 tiles in as many warps."""
    rng = np.random.default_rng(D + hq)
    T = 192
    v = rng.standard_normal((T, hkv, D)) * np.exp2(rng.uniform(-1, 1, (T, 1, 1)))
    check(case(1, rng.integers(0, 13, T).astype(float), v, [1, 3, 7, 16, 20, 33, 60, 100, 130], hq, hkv, P, dt, meta), hkv, P,
          meta, odt)


@pytest.mark.parametrize("D,hq,hkv,P,dt,odt,meta", CASES)
def test_small_products_beside_a_large_scale(D, hq, hkv, P, dt, odt, meta):
    """One value row of 0 and 15 in 16, the others 1.37 2^-13 of it: in the dims of its zeros only the others'
    products count, cut as if they were of its size.  All weights are equal."""
    rng = np.random.default_rng(D + hq)
    T = 192
    v = rng.integers(0, 16, (T, hkv, D)) * (1.37 * 2.0 ** -13)
    v[:, :, :2], v[:, :, 2:4] = 0.0, 15 * 1.37 * 2.0 ** -13  # (zeros of 0)
    at = np.arange(0, T, 16) + rng.integers(0, 3, T // 16)
    v[at] = 15.0 * rng.integers(0, 2, (len(at), hkv, D))
    v[at, :, :2], v[at, :, 2:4] = 0.0, 15.0
    check(case(2, np.zeros(T), v, [16, 32, 100, 130], hq, hkv, P, dt, meta), hkv, P, meta, odt)
