"""Plain numpy forms of a sparse decode step's operators: the norm and the page
summaries step by step in binary32 (numpy rounds every operation once), the
page lists in whole numbers, the attention in 64 bits."""
import numpy as np

import oracle

U = 2.0 ** -24  # a binary32 rounding, relative


def norm_rows(x, w, offset, eps, to=np.float32):
    """Rows [..., D] over the root of their mean square, times the gains (None: without)."""
    x = x.astype(to)
    D = x.shape[-1]
    if to is np.float32:
        t = x * x
        while t.shape[-1] > 1:
            t = t[..., 0::2] + t[..., 1::2]
        r = np.float32(1) / np.sqrt(t * np.float32(1.0 / D) + np.float32(eps))
    else:
        r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + np.float32(eps))
    y = x * r
    return y if w is None else y * (w.astype(to) + to(offset))


def word_value(bits, meta_bf16):
    """{scale, zero} bits (uint16) -> binary32."""
    if meta_bf16:
        return (bits.astype(np.uint32) << 16).view(np.float32)
    return bits.view(np.float16).astype(np.float32)


def quantize(y, meta_bf16):
    """Rows float32 [..., D] -> packed codes [..., D/2] and {scale, zero} bytes [..., 4]."""
    conv = oracle.f32_to_bf16_bits if meta_bf16 else oracle.f32_to_f16_bits
    z = conv(y.min(-1), oracle.RD)
    step = (y.max(-1) - word_value(z, meta_bf16)) / np.float32(15)
    s = conv(step, oracle.RU)
    if meta_bf16:
        s = np.where((step > 0) & (s < 0x80), np.uint16(0x80), s)
    sv, zv = word_value(s, meta_bf16), word_value(z, meta_bf16)
    r = np.divide(np.float32(1), sv, out=np.zeros_like(sv), where=sv != 0)
    q = np.clip(np.rint((y - zv[..., None]) * r[..., None]), 0, 15).astype(np.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), np.stack((s, z), -1).astype(np.uint16).view(np.uint8)


def rows_of(cache, page, head, hkv, D, P, meta_bf16):
    """Codes [P, D], scales [P] and zeros [P] of a page, in binary32."""
    n = P * (D // 2 + 4)
    c = cache[(page * hkv + head) * n:(page * hkv + head + 1) * n]
    q = c[:P * D // 2].reshape(P, D // 2)
    code = np.empty((P, D), np.float32)
    code[:, 0::2], code[:, 1::2] = q & 15, q >> 4
    w = word_value(c[P * D // 2:].copy().view(np.uint16).reshape(P, 2), meta_bf16)
    return code, w[:, 0], w[:, 1]


def summary_stride(hkv, D):
    return (hkv * (D // 2 + 4) + 15) // 16 * 16


def summary_rows(summary, hkv, D):
    """Views of the summaries: packed codes [pages, hkv, D/2], {scale, zero} bytes [pages, hkv, 4]."""
    x = summary.reshape(-1, summary_stride(hkv, D))
    return (x[:, :hkv * D // 2].reshape(-1, hkv, D // 2),
            x[:, hkv * D // 2:hkv * (D // 2 + 4)].reshape(-1, hkv, 4))


def put_summary(summary, page, head, codes, words, hkv, D):
    row = summary.reshape(-1, summary_stride(hkv, D))[page]
    row[head * D // 2:(head + 1) * D // 2] = codes
    row[hkv * D // 2 + 4 * head:hkv * D // 2 + 4 * head + 4] = words


def page_mean(cache, page, head, hkv, D, P, meta_bf16):
    """The mean key of a page by the rule, in binary32."""
    code, s, z = rows_of(cache, page, head, hkv, D, P, meta_bf16)
    a, b = np.zeros((2, D), np.float32), np.zeros(2, np.float32)
    for t in range(P):
        a[t & 1] += code[t] * s[t]
        b[t & 1] += z[t]
    return ((a[0] + a[1]) + (b[0] + b[1])) * np.float32(1.0 / P)


def summaries(summary, cache, bt, lens, new, hkv, D, P, meta_bf16):
    """Writes the rule's summaries of every page that the new tokens completed."""
    for b, L in enumerate(lens):
        n = L if new is None else min(new[b], L)
        for e in range((L - n) // P, L // P):
            for h in range(hkv):
                c, w = quantize(page_mean(cache, bt[b][e], h, hkv, D, P, meta_bf16), meta_bf16)
                put_summary(summary, bt[b][e], h, c, w, hkv, D)


def page_scores(q, summary, ids, group, D, rotate, h, meta_bf16):
    """Scores [hkv, len(ids)] of these pages for q [Hq, D] (float32), step by step."""
    hkv = q.shape[0] // group
    y = oracle.rotate_canon(q, h) if rotate else q
    with np.errstate(all="ignore"):
        top = np.abs(y).max(-1)
        qs = top / np.float32(127)
        r = np.where(qs < np.float32(2.0 ** -126), np.float32(0), np.float32(1) / qs)
        m = np.clip(np.rint(y * r[:, None]), -127, 127)
        codes, words = summary_rows(summary, hkv, D)
        ok = (ids >= 0) & (ids < codes.shape[0])
        at = np.where(ok, ids, 0)
        n = np.empty((len(at), hkv, D), np.float64)
        n[..., 0::2], n[..., 1::2] = codes[at] & 15, codes[at] >> 4
        w = word_value(words[at].copy().view(np.uint16), meta_bf16)
        out = np.empty((hkv, len(ids)), np.float32)
        for k in range(hkv):
            best = np.full(len(ids), -np.inf, np.float32)
            for i in range(k * group, (k + 1) * group):
                dot = (n[:, k] @ m[i].astype(np.float64)).astype(np.float32)  # whole, below 2^24
                sc = qs[i] * (w[:, k, 0] * dot + w[:, k, 1] * np.float32(m[i].sum()))
                best = np.maximum(best, np.where(np.isnan(sc), np.float32(-np.inf), sc))
            out[k] = np.where(ok, best, np.float32(-np.inf)) + np.float32(0)
    return out


def select(q, summary, bt, lens, hkv, D, P, rotate, h, take, first, last, meta_bf16):
    """(tables, pages, lens) of every (sequence, kv-head)."""
    B, G = len(lens), q.shape[1] // hkv
    tables, pages = np.full((2, B, hkv, take), -1, np.int32)
    out = np.zeros((B, hkv), np.int32)
    for b, L in enumerate(lens):
        n = -(-int(L) // P)
        if n > take:
            sc = page_scores(q[b], summary, bt[b][first:n - last], G, D, rotate, h, meta_bf16)
        for k in range(hkv):
            e = np.arange(n)
            if n > take:
                order = np.lexsort((np.arange(sc.shape[1]), -sc[k]))[:take - first - last]
                e = np.concatenate((e[:first], first + np.sort(order), e[n - last:]))
            tables[b, k, :len(e)], pages[b, k, :len(e)] = bt[b][e], e
            out[b, k] = len(e) * P - (n * P - L)
    return tables, pages, out


def matrix(h, D):
    m = np.ones((1, 1))
    while m.shape[0] < h:
        m = np.block([[m, m], [m, -m]])
    return np.kron(np.eye(D // h), m / np.sqrt(h))


def attend(q, kc, vc, tables, lens, hkv, D, P, rot_k, rot_v, h, scale, meta_bf16, pages):
    """Attention in 64 bits over the listed pages (a bad page is passed over), the
    largest row norm of the values, and per row the standard deviation of an
    output's error when each p s is rounded to 11 bits: sqrt(sum (p |s n|)^2)
    2^-11 / sqrt 3 bounds that of any one output, rotated back or not."""
    B, Hq, _ = q.shape
    G, H = Hq // hkv, matrix(h, D)
    out, sd, top = np.zeros((B, Hq, D)), np.zeros((B, Hq)), 0.0
    for b in range(B):
        for k in range(hkv):
            L = int(lens[b, k])
            ks, vs, ns = [], [], []
            for e in range(-(-L // P)):
                page = int(tables[b, k, e])
                if not 0 <= page < pages:
                    continue
                t = min(P, L - e * P)
                (ck, sk, zk), (cv, sv, zv) = (rows_of(c, page, k, hkv, D, P, meta_bf16) for c in (kc, vc))
                ks.append((ck.astype(np.float64) * sk[:, None] + zk[:, None])[:t])
                vs.append((cv.astype(np.float64) * sv[:, None] + zv[:, None])[:t])
                ns.append((cv.astype(np.float64) * sv[:, None])[:t])
            if not ks:
                continue
            K, V, N = (np.concatenate(x) for x in (ks, vs, ns))
            top = max(top, np.sqrt((V * V).sum(-1)).max())
            x = q[b, k * G:(k + 1) * G].astype(np.float64)
            lg = (x @ H if rot_k else x) @ K.T * scale
            p = np.exp(lg - lg.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            o = p @ V
            out[b, k * G:(k + 1) * G] = o @ H if rot_v else o
            sd[b, k * G:(k + 1) * G] = np.sqrt((p * p) @ (N * N).sum(-1)) * 2.0 ** -11 / np.sqrt(3)
    return out, top, sd
