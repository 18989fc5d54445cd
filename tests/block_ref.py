"""Plain numpy restatements of the attention half's operators (include/zdmmv.h): the cache's layout, the Q4_0 and
Q8_0 blocks, the rotation in fp32 operation by operation, the norm and the attention in 64 bits."""
import numpy as np

QK, SLAB = 32, 16


def tile_index(dim):
    """(K nibble, V nibble, scale) numbers of a tile's values: [16][dim], [16][dim], [16][dim/32]; word by word from
    the header's formulas."""
    nb = dim // QK
    w = 4 if nb % 4 == 0 else 2 if nb % 2 == 0 else 1
    k, v, s = (np.zeros((SLAB, n), dtype=np.int64) for n in (dim, dim, nb))
    for r in range(SLAB):
        for b in range(nb):
            s[r, b] = ((r // 2) * nb + b) * 2 + r % 2
            for f in range(QK):
                word = (((r // 8) * (nb // w) + b // w) * 32 + (r % 8) * 4 + f // 8) * w + b % w
                k[r, QK * b + f] = 8 * word + f % 8
                word = (((r // 8) * (nb // w) + b // w) * 32 + (f // 4) * 4 + (r % 8) // 2) * w + b % w
                v[r, QK * b + f] = 8 * word + 4 * (r % 2) + f % 4
    return k, v, s


def unpack(pages, page_tokens, heads, dim):
    """uint8 pages -> (K codes, V codes, K scales, V scales): codes int [page][head][token][dim] as code - 8, scales
    fp16 [page][head][token][dim/32]."""
    t = np.ascontiguousarray(pages).reshape(-1, heads, page_tokens // SLAB, 18 * dim)
    ik, iv, isc = tile_index(dim)
    out = []
    for base, i in ((0, ik), (8 * dim, iv)):
        nib = np.stack((t[..., base:base + 8 * dim] & 15, t[..., base:base + 8 * dim] >> 4), -1)
        nib = nib.reshape(*t.shape[:3], -1)
        out.append((nib[..., i].astype(np.int32) - 8).reshape(t.shape[0], heads, page_tokens, dim))
    for base in (16 * dim, 17 * dim):
        h = np.ascontiguousarray(t[..., base:base + dim]).view(np.float16)
        out.append(h[..., isc].reshape(t.shape[0], heads, page_tokens, dim // QK))
    return out


def values(pages, page_tokens, heads, dim):
    """fp64 K and V, [page][head][token][dim]."""
    kc, vc, kd, vd = unpack(pages, page_tokens, heads, dim)
    with np.errstate(invalid="ignore"):
        return [c * np.repeat(d.astype(np.float64), QK, -1) for c, d in ((kc, kd), (vc, vd))]


def put(pages, page_tokens, heads, dim, page, tok, head, which, codes, scales):
    """Write one token's codes (0..15, [dim]) and fp16 scales ([dim/32]) of one head into pages (uint8, in place);
    which: 0 K, 1 V."""
    i = tile_index(dim)
    t = pages.reshape(-1, heads, page_tokens // SLAB, 18 * dim)[page, head, tok // SLAB]
    n = i[which][tok % SLAB]
    c = t[8 * dim * which:8 * dim * (which + 1)]
    for j in range(dim):
        byte, high = n[j] // 2, n[j] % 2
        c[byte] = (c[byte] & (0x0F if high else 0xF0)) | (int(codes[j]) << (4 if high else 0))
    base = (16 + which) * dim
    h = t[base:base + dim].view(np.float16)
    h[i[2][tok % SLAB]] = scales


def quantize_q4(x):
    """Q4_0 of fp32 rows [..., dim] in fp32 operations: (codes 0..15 [..., dim], fp16 scales [..., dim/32])."""
    b = np.asarray(x, np.float32).reshape(-1, QK)
    at = np.argmax(np.abs(b), 1)  # the first of the largest magnitude
    d = (b[np.arange(len(b)), at] / np.float32(-8)).astype(np.float32)
    with np.errstate(divide="ignore"):
        inv = np.where(d != 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
    q = np.minimum(np.trunc((b * inv[:, None]).astype(np.float32) + np.float32(8.5)), 15).astype(np.int32)
    return q.reshape(x.shape), d.astype(np.float16).reshape(*x.shape[:-1], -1)


def rotate(x, table, pos, halves):
    """fp32 rotation of [tok][head][dim] by rows `pos` of table [n][rot], every product and sum rounded."""
    x = np.array(x, np.float32)
    rot = table.shape[1]
    h = rot // 2
    c, s = table[pos][:, None, :h].astype(np.float32), table[pos][:, None, h:].astype(np.float32)
    ia, ib = (slice(0, h), slice(h, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = a * s + b * c
    return x


def rope_table(n, rot, base=10000.0):
    angle = np.arange(n)[:, None] * base ** (-np.arange(rot // 2) * 2.0 / rot)
    return np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32)


def attention(q, q_start, kv_len, table, k, v, page_tokens, scale, window=0):
    """fp64 attention of q [tok][heads][dim] over k, v ([page][head][token][dim] values). Returns (out, tol_p, tol_v):
    tol_p [tok][head] = scale * max_t sum_e |q_e| * (8 / 7.5 of the largest |k| magnitudes' bound), used by the tests'
    error bound, and tol_v [tok][head][dim] = sum_t p_t * max|v_t's block|."""
    n_tok, hq, dim = q.shape
    hk = k.shape[1]
    out = np.zeros(q.shape)
    tol_p, tol_v = np.zeros((n_tok, hq)), np.zeros(q.shape)
    for s in range(len(kv_len)):
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            row = q_start[s] + i
            end = kv_len[s] - (n - 1 - i)
            low = max(0, end - window) if window else 0
            if end <= low:
                continue
            t = np.arange(low, end)
            page, at = table[s][t // page_tokens], t % page_tokens
            for h in range(hq):
                kk, vv = k[page, h // (hq // hk), at], v[page, h // (hq // hk), at]
                score = kk @ q[row, h].astype(np.float64) * scale
                p = np.exp(score - score.max())
                p /= p.sum()
                out[row, h] = p @ vv
                big_k = np.abs(kk).reshape(len(t), -1, QK).max(-1)
                big_v = np.abs(vv).reshape(len(t), -1, QK).max(-1)
                tol_p[row, h] = abs(scale) * (big_k @ np.abs(q[row, h]).reshape(-1, QK).sum(-1)).max()
                tol_v[row, h] = np.repeat(p @ big_v, QK)
    return out, tol_p, tol_v
