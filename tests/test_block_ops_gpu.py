"""The attention half's operators on the GPU against plain numpy restatements (tests/block_ref.py).

Bounds (u = 2^-24, fp32's half unit):
  norm       s bit for bit. y's relative error is below e = 100 u: the sum of squares adds at most 128 terms in a
             chain and 12 levels of a tree (half of their 140 u counts in the root), and six roundings follow; then a
             code is within 0.5 + 254 e of y / d, the scale within fp16's half unit and e of it.
  append     bit for bit: every operation is a rounded fp32 operation with one result.
  attention  K's and V's codes are exact in fp16; q and p are split in two fp16 parts (2^-22 of the value). A score
             adds products of at most 8 blocks of 32 with sums that stay below 16 |d q| a term: its error is below
             2^-19 P, P = scale * sum |q_e| max|k_block|; p's and so the result's relative error is twice that. The
             sums over the tokens add below 2^-17 of sum p max|v_block| for up to 4096 tokens (64 steps of 2^-23 for
             each of the parts that are joined).
"""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("rows, cols", [(1, 32), (1, 64), (3, 96), (1, 2048), (8, 4096), (5, 1312), (301, 128),
                                        (2, 5120), (1, 8192), (3, 11008), (2, 32768), (1, 32736), (4099, 32)])
@pytest.mark.parametrize("residual, weight", [(True, True), (False, False)])
def test_norm(rows, cols, residual, weight):
    rng = np.random.default_rng(rows * 7 + cols)
    x = (rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-8, 8, (rows, 1)))).astype(np.float32)
    r = rng.standard_normal((rows, cols)).astype(np.float32) if residual else None
    w = (1 + 0.2 * rng.standard_normal(cols)).astype(np.float32) if weight else None
    x[0, :32] = 0
    if residual:
        r[0, :32] = 0          # a block of zeros
    xd = dev(x)
    out, y = torch.full((rows, cols), float("nan"), device="cuda"), torch.full((rows, cols), float("nan"), device="cuda").half()
    xq = torch.full((rows * cols // 32 * 34 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    Z.add_rmsnorm_q8_0(xd, None if w is None else dev(w), 1e-5, residual=None if r is None else dev(r), out=out, xq=xq, y=y)
    s = x + r if residual else x
    assert np.array_equal(out.cpu().numpy(), s)
    raw = xq.cpu().numpy()
    assert np.all(raw[rows * cols // 32 * 34:] == 0xA5)
    blocks = raw[:rows * cols // 32 * 34].reshape(-1, 34)
    d = np.ascontiguousarray(blocks[:, :2]).view(np.float16)[:, 0].astype(np.float64)
    q = blocks[:, 2:].view(np.int8).astype(np.float64)
    s64 = s.astype(np.float64)
    want = s64 / np.sqrt((s64 * s64).mean(1, keepdims=True) + 1e-5)
    want = (want * (1 if w is None else w.astype(np.float64))).reshape(-1, 32)
    step = np.abs(want).max(1) / 127
    e = 100 * U
    assert np.all(np.abs(d - step) <= step * (2.0 ** -11 + e) + 2.0 ** -25)
    ratio = np.divide(want, step[:, None], out=np.zeros_like(want), where=step[:, None] > 0)
    assert np.all(np.abs(q - ratio) <= 0.5 + 254 * e)
    assert np.array_equal(y.cpu().numpy().reshape(-1, 32), (q * d[:, None]).astype(np.float16))


def test_norm_strided_and_in_place():
    rng = np.random.default_rng(5)
    big = dev(rng.standard_normal((9, 700)).astype(np.float32))
    x, r = big[:, 4:644], dev(rng.standard_normal((9, 640)).astype(np.float32))
    want = Z.add_rmsnorm_q8_0(x.contiguous(), None, 1e-6, residual=r)
    out = torch.empty(9, 640, device="cuda")
    assert torch.equal(Z.add_rmsnorm_q8_0(x, None, 1e-6, residual=r, out=out), want)
    for target in ("x", "r"):
        xc, rc = x.contiguous(), r.clone()
        got = Z.add_rmsnorm_q8_0(xc, None, 1e-6, residual=rc, out=xc if target == "x" else rc)
        assert torch.equal(got, want) and torch.equal(xc if target == "x" else rc, out)
    # outputs that are not asked for stay unwritten, and the others are the same
    y = torch.empty(9, 640, dtype=torch.float16, device="cuda")
    assert torch.equal(Z.add_rmsnorm_q8_0(x, None, 1e-6, residual=r, y=y), want)


def test_norm_feeds_the_dmmv():
    """The blocks are those that zdmmv_quantize_act_q8_0 forms of the same values: a row whose norm is exact."""
    x = torch.zeros(1, 2048, device="cuda")
    x[0, ::2], x[0, 1::2] = 1.0, -1.0                      # mean square 1
    w = torch.randn(2048, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    xq = Z.add_rmsnorm_q8_0(x, w, 1e-30)
    assert torch.equal(xq, Z.quantize_act_q8_0((x[0] * w).contiguous()))


# ------------------------------------------------------------------ append
def make_cache(n_pages, page, heads, dim, table, fill=None, seed=0):
    n = n_pages * Z.kv_page_bytes(page, heads, dim)
    pages = np.random.default_rng(seed).integers(0, 256, n, dtype=np.uint8) if fill is None else np.full(n, fill, np.uint8)
    t = dev(np.asarray(table, np.int32))
    return Z.KVCache(dev(pages), page, heads, dim, t), pages


@pytest.mark.parametrize("dim, rot, halves", [(64, 64, True), (64, 34, False), (96, 96, False), (128, 128, True),
                                              (128, 128, False), (128, 50, True), (192, 64, True), (256, 256, True),
                                              (256, 64, False), (128, 0, True)])
@pytest.mark.parametrize("page, heads, group", [(16, 1, 1), (48, 3, 5), (64, 2, 8)])
def test_append(dim, rot, halves, page, heads, group):
    rng = np.random.default_rng(dim + rot + page)
    n_seq, max_pages, n_pages = 3, 4, 13
    table = rng.permutation(n_pages)[:12].reshape(n_seq, max_pages)
    cache, pages = make_cache(n_pages, page, heads, dim, table)
    # a padded token, a token of the last position, pages' first and last tokens, the others in any order
    seq = np.array([0, 1, 2, 2, 0, 1, 1, 0], np.int32)
    pos = np.array([0, -1, max_pages * page - 1, page - 1, page, 17, 2 * page + 15, 5], np.int32)
    n = len(seq)
    hq = heads * group
    joint = (rng.standard_normal((n, (hq + 2 * heads) * dim)) * np.exp2(rng.integers(-6, 6, (n, 1)))).astype(np.float32)
    joint[4, (hq + heads) * dim:] = 0                       # a token of zeros
    joint[5, hq * dim] = joint[5, hq * dim + 1] * -1        # magnitudes that tie
    jd = dev(joint)
    q, k, v = jd[:, :hq * dim], jd[:, hq * dim:(hq + heads) * dim], jd[:, (hq + heads) * dim:]
    rope = R.rope_table(max_pages * page, rot) if rot else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kval, vval = (torch.full((n, heads, dim), float("nan"), device="cuda").half() for _ in range(2))
    style = Z.ROPE_HALVES if halves else Z.ROPE_PAIRS
    qo = Z.kv_append_q4_0(cache, k, v, dev(seq), dev(pos), q=q, rope=None if rope is None else dev(rope), rope_style=style,
                          k_val=kval, v_val=vval, status=status)
    x = joint.reshape(n, hq + 2 * heads, dim)
    live = pos >= 0
    turned = x[:, :hq + heads].copy()
    if rot:
        turned[live] = R.rotate(turned[live], rope, pos[live], halves)
    want_q = np.where(live[:, None, None], turned[:, :hq], 0)
    assert np.array_equal(qo.cpu().numpy(), want_q)
    want = pages.copy()
    for which, rows, val in ((0, turned[:, hq:], kval), (1, x[:, hq + heads:], vval)):
        code, d = R.quantize_q4(rows)
        for t in range(n):
            for h in range(heads if live[t] else 0):
                R.put(want, page, heads, dim, table[seq[t], pos[t] // page], pos[t] % page, h, which, code[t, h], d[t, h])
        stands = ((code - 8) * np.repeat(d.astype(np.float32), 32, -1)).astype(np.float16)
        assert np.array_equal(val.cpu().numpy(), np.where(live[:, None, None], stands, 0))
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    assert status.item() == 0
    # q in place, and without q, without values: the same cache
    q2 = q.contiguous()
    Z.kv_append_q4_0(cache, k, v, dev(seq), dev(pos), q=q2, q_out=q2, rope=None if rope is None else dev(rope), rope_style=style)
    assert torch.equal(q2.view_as(qo), qo)
    c2, _ = make_cache(n_pages, page, heads, dim, table)
    Z.kv_append_q4_0(c2, k.contiguous(), v.view(n, heads, dim), dev(seq), dev(pos),
                     rope=None if rope is None else dev(rope), rope_style=style)
    assert torch.equal(c2.pages, cache.pages)


@pytest.mark.parametrize("dim, rot, halves", [(64, 64, True), (96, 50, True), (128, 128, True), (128, 64, False),
                                              (192, 128, True), (256, 256, True), (256, 34, False)])
@pytest.mark.parametrize("heads, group", [(2, 4), (1, 1), (3, 1)])
def test_append_prompt(dim, rot, halves, heads, group):
    """Many tokens at once (the kernel for prompts) are the same tokens a few at a time, byte for byte: two sequences, a
    padded stretch, bad tokens among the good ones."""
    n = -(-12000 // (heads * (group + 2)))
    page, n_seq = 48, 2
    max_pages = -(-n // page)
    rng = np.random.default_rng(n + dim)
    table = rng.permutation(2 * max_pages).reshape(n_seq, max_pages)
    table[1, 3] = 1 << 28
    seq = (np.arange(n) % 2).astype(np.int32)
    pos = (np.arange(n) // 2).astype(np.int32)
    pos[100:117] = -1
    seq[200] = 2
    hq = heads * group
    g = torch.Generator("cuda").manual_seed(n)
    joint = torch.randn(n, (hq + 2 * heads) * dim, device="cuda", generator=g)
    q, k, v = joint[:, :hq * dim], joint[:, hq * dim:(hq + heads) * dim], joint[:, (hq + heads) * dim:]
    rope, seq, pos = dev(R.rope_table(max_pages * page, rot)), dev(seq), dev(pos)
    style = Z.ROPE_HALVES if halves else Z.ROPE_PAIRS

    def run(step):
        cache, _ = make_cache(2 * max_pages, page, heads, dim, table)
        vals = [torch.empty(n, heads, dim, dtype=torch.float16, device="cuda") for _ in range(2)]
        out, status = torch.empty(n, hq, dim, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        for i in range(0, n, step):
            s = slice(i, min(n, i + step))
            Z.kv_append_q4_0(cache, k[s], v[s], seq[s], pos[s], q=q[s], q_out=out[s], rope=rope, rope_style=style,
                             k_val=vals[0][s], v_val=vals[1][s], status=status)
        return cache.pages, out, *vals, status
    once, pieces = run(n), run(97)
    assert once[4].item() == 1
    for a, b in zip(once, pieces):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert Z.device_status() == 0


def test_append_bad_tokens():
    page, heads, dim = 16, 2, 128
    table = np.array([[0, 1], [-1, 5], [2, 3]])
    cache, pages = make_cache(4, page, heads, dim, table)
    seq = np.array([-1, 3, 0, 1, 1, 2, 2], np.int32)        # sequences, positions and pages out of range ...
    pos = np.array([0, 0, 32, 3, 17, 40000, 20], np.int32)  # ... and one good token
    g = torch.Generator("cuda").manual_seed(1)
    k, v, q = (torch.randn(7, heads * dim, device="cuda", generator=g) for _ in range(3))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kval = torch.zeros(7, heads, dim, dtype=torch.float16, device="cuda")
    rope = dev(R.rope_table(64, dim))
    qo = Z.kv_append_q4_0(cache, k, v, dev(seq), dev(pos), q=q, rope=rope, k_val=kval, status=status)
    assert status.item() == 1
    assert qo[:6].isnan().all() and not qo[6].isnan().any()
    assert kval[:6].isnan().all() and not kval[6].isnan().any()
    now = cache.pages.cpu().numpy().reshape(4, -1)
    assert np.array_equal(now[:3], pages.reshape(4, -1)[:3])
    # a position past the rotation's rows is bad too
    status.zero_()
    Z.kv_append_q4_0(cache, k[:1], v[:1], dev(seq[6:]), dev(np.array([20], np.int32)), rope=rope[:20], status=status)
    assert status.item() == 1 and np.array_equal(cache.pages.cpu().numpy().reshape(4, -1), now)


# ------------------------------------------------------------------ attention
def random_cache(rng, lens, page, heads, dim, spare=1, dead=None):
    """Pages in any order for sequences of these lengths: random codes, scales of both signs. dead: what the bytes of
    the pages' unused tokens (and of the pages nobody holds) are."""
    held = [max(0, -(-n // page)) for n in lens]
    max_pages = max(1, max(held)) + spare
    n_pages = sum(held) + 2
    order = list(rng.permutation(n_pages))
    table = np.full((len(lens), max_pages), -1, np.int32)
    cache, pages = make_cache(n_pages, page, heads, dim, table, fill=0xFF if dead is None else dead)
    t = pages.reshape(n_pages, heads, page // 16, 18 * dim)
    ik, iv, isc = R.tile_index(dim)
    for s, n in enumerate(lens):
        for i in range(held[s]):
            p = order.pop()
            table[s, i] = p
            for j in range(page // 16):
                live = min(16, n - i * page - j * 16)
                if live <= 0:
                    continue
                fresh = rng.integers(0, 256, (heads, 18 * dim), dtype=np.uint8)
                sc = (rng.uniform(0.05, 0.3, (heads, dim)) * rng.choice([-1, 1], (heads, dim))).astype(np.float16)
                fresh[:, 16 * dim:] = sc.view(np.uint8)
                keep = np.zeros(18 * dim, bool)   # bytes of the tile's live tokens
                for base, idx in ((0, ik), (8 * dim, iv)):
                    keep[base + idx[:live].ravel() // 2] = True
                for base in (16 * dim, 17 * dim):
                    keep[base + 2 * isc[:live].ravel()] = True
                    keep[base + 2 * isc[:live].ravel() + 1] = True
                t[p, :, j] = np.where(keep, fresh, t[p, :, j])
    return Z.KVCache(dev(pages), page, heads, dim, dev(table)), pages, table


def check_attention(out, q, q_start, lens, table, pages, page, heads, dim, scale=None, window=0):
    scale = dim ** -0.5 if scale is None else scale
    k, v = R.values(pages, page, heads, dim)
    want, tp, tv = R.attention(q, q_start, lens, table, k, v, page, scale, window)
    got = out.double().cpu().numpy()
    tol = tv * (2 * 2.0 ** -19 * tp + 2.0 ** -17)[..., None]
    assert np.isfinite(got).all()
    bad = np.abs(got - want) - tol
    assert (bad <= 0).all(), (bad.max(), np.abs(got - want).max(), np.unravel_index(bad.argmax(), bad.shape))


def run_attention(rng, lens, new, page, heads, group, dim, window=0, scale=None, dead=None, sharp=1.5):
    cache, pages, table = random_cache(rng, lens, page, heads, dim, dead=dead)
    q_start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = (sharp * rng.standard_normal((q_start[-1], heads * group, dim))).astype(np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), device="cuda")
    Z.attn_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), max(new), max(lens), scale=scale, window=window,
                out=out, status=status)
    assert status.item() == 0
    check_attention(out, q, q_start, lens, table, pages, page, heads, dim, scale, window)
    return cache, q, q_start, out


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads, group", [(1, 1), (2, 4), (1, 8), (2, 5), (1, 16), (1, 24)])
def test_attention_one_token(dim, heads, group):
    rng = np.random.default_rng(dim + heads + group)
    run_attention(rng, [1, 16, 37, 300, 1029], [1] * 5, 32, heads, group, dim)


@pytest.mark.parametrize("lens", [[1], [2], [15], [16], [17], [31, 32, 33], [63, 64, 65, 0, 127, 128, 129], [0], [0, 0, 5],
                                  [4093], [255, 256, 257, 2050]])
@pytest.mark.parametrize("page", [16, 48, 64, 1024])
def test_attention_lengths(lens, page):
    run_attention(np.random.default_rng(sum(lens) + page), lens, [1] * len(lens), page, 2, 4, 128)


@pytest.mark.parametrize("lens, new, window", [
    ([5], [5], 0), ([700, 33, 8], [8, 3, 8], 0), ([700, 33, 8], [2, 7, 1], 16), ([1000, 129], [1, 1], 1),
    ([1000, 129], [4, 4], 100), ([3, 40, 0], [6, 2, 2], 0),        # more new tokens than the cache holds: empty rows
    ([600, 50], [70, 50], 0), ([1500], [130], 33), ([90, 1111, 64], [0, 65, 64], 0), ([333], [333], 0)])
@pytest.mark.parametrize("heads, group, dim", [(2, 4, 128), (3, 1, 64), (1, 7, 256), (1, 16, 96)])
def test_attention_new_tokens(lens, new, window, heads, group, dim):
    run_attention(np.random.default_rng(sum(lens) + sum(new) + window), lens, new, 32, heads, group, dim, window=window)


def ragged(rng, n, most):
    """Lengths from 0 and 1 to `most`, most of them short."""
    lens = np.exp(rng.uniform(0, np.log(most), n)).astype(int)
    lens[:3] = most, 0, 1
    return rng.permutation(lens).tolist()


@pytest.mark.parametrize("n_seq, most, heads, group, dim, window", [
    (40, 4000, 8, 4, 128, 0), (40, 4000, 8, 1, 128, 900), (24, 5000, 8, 8, 128, 0), (90, 3000, 4, 16, 64, 0),
    (28, 3500, 6, 12, 256, 0), (60, 2000, 6, 3, 96, 0), (40, 3000, 4, 8, 192, 0)])
def test_attention_many_long_sequences(n_seq, most, heads, group, dim, window):
    """Enough steps that the CTAs take stretches of all sequences' steps: shared items, whole ones, empty ones."""
    rng = np.random.default_rng(n_seq + most)
    lens = ragged(rng, n_seq, most)
    cache, q, q_start, out = run_attention(rng, lens, [1] * n_seq, 64, heads, group, dim, window=window)
    for _ in range(3):  # the same bits again
        again = Z.attn_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), 1, most, window=window)
        assert torch.equal(again, out)


def test_attention_more_sequences_than_threads():
    """More than 256 sequences, some with two new tokens, some with none, a bad one among them."""
    rng = np.random.default_rng(21)
    n_seq, heads, group, dim, page = 700, 2, 2, 128, 32
    lens = ragged(rng, n_seq, 760)
    new = [int(min(n, rng.integers(0, 3))) for n in lens]
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    q_start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = rng.standard_normal((q_start[-1], heads * group, dim)).astype(np.float32)
    bad = next(s for s in range(300, n_seq) if new[s])
    now = np.array(lens, np.int32)
    now[bad] = -5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Z.attn_q4_0(cache, dev(q), dev(q_start), dev(now), 2, 760, status=status)
    rows = slice(q_start[bad], q_start[bad + 1])
    assert status.item() == 1 and out[rows].isnan().all()
    keep = np.setdiff1d(np.arange(q_start[-1]), np.arange(rows.start, rows.stop))
    k, v = R.values(pages, page, heads, dim)
    want, tp, tv = R.attention(q, q_start, lens, table, k, v, page, dim ** -0.5)
    got = out.double().cpu().numpy()
    tol = tv * (2 * 2.0 ** -19 * tp + 2.0 ** -17)[..., None]
    assert (np.abs(got - want) <= tol)[keep].all()


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("new, lens, window", [([40, 3], [1200, 300], 0), ([150], [4000], 0), ([64], [64], 20)])
def test_attention_prompts(dim, new, lens, window):
    run_attention(np.random.default_rng(dim + sum(new)), lens, new, 48, 2, 4, dim, window=window)


def test_attention_windows_read_no_older_page():
    """Pages wholly before the window may be gone."""
    rng = np.random.default_rng(9)
    page, heads, group, dim, window = 32, 2, 4, 128, 70
    cache, pages, table = random_cache(rng, [500, 230], page, heads, dim)
    gone = table.copy()
    for s, n in enumerate((500, 230)):
        gone[s, :(n - 3 - window) // page] = -1
    cache.page_table.copy_(dev(gone))
    q = rng.standard_normal((6, heads * group, dim)).astype(np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_start, lens = np.array([0, 3, 6], np.int32), np.array([500, 230], np.int32)
    out = Z.attn_q4_0(cache, dev(q), dev(q_start), dev(lens), 3, 500, window=window, status=status)
    assert status.item() == 0
    check_attention(out, q, q_start, lens, table, pages, page, heads, dim, window=window)


@pytest.mark.parametrize("sharp, scale", [(30.0, None), (0.0, None), (1.0, 0.0), (1.0, -0.3), (1e-20, 1.0), (1e4, 1e-3)])
def test_attention_scores_of_any_size(sharp, scale):
    run_attention(np.random.default_rng(3), [777, 60], [1, 2], 16, 2, 4, 128, scale=scale, sharp=sharp)


def test_attention_scales_of_any_size():
    """Rows whose blocks' scales span fp16's range, and zero blocks."""
    rng = np.random.default_rng(4)
    page, heads, group, dim, lens = 16, 1, 4, 128, [400]
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    t = pages.reshape(-1, 18 * dim)
    for which, lo, hi in ((16, -14, -2), (17, -24, 12)):
        sc = (np.exp2(rng.uniform(lo, hi, (len(t), dim // 2))) * rng.choice([-1, 0, 1], (len(t), dim // 2))).astype(np.float16)
        t[:, which * dim:(which + 1) * dim] = sc.view(np.uint8)
    cache.pages.copy_(dev(pages))
    q = rng.standard_normal((1, 4, dim)).astype(np.float32)
    out = Z.attn_q4_0(cache, dev(q), dev(np.array([0, 1], np.int32)), dev(np.array(lens, np.int32)), 1, 400)
    check_attention(out, q, [0, 1], lens, table, pages, page, heads, dim)


def test_attention_exact_sums():
    """q = 0: every p is 1, so with scales of 1 the result is a mean of small integers, and exact for powers of two."""
    rng = np.random.default_rng(6)
    page, heads, group, dim = 64, 2, 4, 128
    lens = [1, 64, 512, 2048]
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    t = pages.reshape(-1, 18 * dim)
    t[:, 16 * dim:] = np.ones((len(t), dim), np.float16).view(np.uint8)
    cache.pages.copy_(dev(pages))
    q = np.zeros((4, heads * group, dim), np.float32)
    out = Z.attn_q4_0(cache, dev(q), dev(np.arange(5, dtype=np.int32)), dev(np.array(lens, np.int32)), 1, 2048)
    k, v = R.values(pages, page, heads, dim)
    want, _, _ = R.attention(q, list(range(5)), lens, table, k, v, page, 1.0)
    assert np.array_equal(out.double().cpu().numpy(), want)


def test_attention_bad_sequences():
    rng = np.random.default_rng(7)
    page, heads, group, dim = 16, 2, 4, 128
    lens = [40, 40, 40, 40, 40]
    cache, pages, table = random_cache(rng, lens, page, heads, dim, spare=0)
    bad = table.copy()
    bad[1, 1], bad[2, 0] = 1 << 20, -3
    cache.page_table.copy_(dev(bad))
    now = np.array([40, 40, 40, 49, -2], np.int32)          # 3: past its pages; 4: negative
    q = rng.standard_normal((5, heads * group, dim)).astype(np.float32)
    for order in (np.arange(5), np.arange(5)[::-1].copy()):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = Z.attn_q4_0(cache, dev(q), dev(np.arange(6, dtype=np.int32)), dev(now), 1, 64, status=status)
        assert status.item() == 1
        assert out[1:].isnan().all()
        check_attention(out[:1], q[:1], [0, 1], lens[:1], table[:1], pages, page, heads, dim)
    # more tokens than the call said: the covered rows are NaN; the good sequence keeps its result
    for kw in (dict(max_q_len=1, max_kv_len=64), dict(max_q_len=4, max_kv_len=30)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.zeros(5, heads * group, dim, device="cuda")
        now = np.array([25, 40, 0, 0, 0], np.int32)
        cache.page_table.copy_(dev(table))
        Z.attn_q4_0(cache, dev(q), dev(np.array([0, 1, 5, 5, 5, 5], np.int32)), dev(now), out=out, status=status, **kw)
        assert status.item() == 1 and out[1].isnan().all()
        k, v = R.values(pages, page, heads, dim)
        check_attention(out[:1], q[:1], [0, 1], [25], table[:1], pages, page, heads, dim)


def test_attention_strides_streams_graphs_and_repeats():
    rng = np.random.default_rng(8)
    page, heads, group, dim = 32, 2, 4, 128
    lens = [900, 31]
    cache, q, q_start, out = run_attention(rng, lens, [1, 1], page, heads, group, dim)
    wide = torch.zeros(2, heads * group * dim + 12, device="cuda")
    wide[:, :-12] = dev(q).view(2, -1)
    qs, kv = dev(q_start), dev(np.array(lens, np.int32))
    assert torch.equal(Z.attn_q4_0(cache, wide[:, :-12], qs, kv, 1, 900), out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = Z.attn_q4_0(cache, dev(q), qs, kv, 1, 900, stream=side)
    side.synchronize()
    assert torch.equal(got, out)
    # a captured call replays with new lengths within its bounds
    q2, o2 = dev(q), torch.empty_like(out)
    ws = Z.attn_q4_0_workspace(cache, heads * group, 1, 900)
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            Z.attn_q4_0(cache, q2, qs, kv, 1, 900, out=o2, workspace=ws)
    for new in ([900, 31], [17, 2], [640, 0]):
        kv.copy_(dev(np.array(new, np.int32)))
        for _ in range(2):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, Z.attn_q4_0(cache, q2, qs, kv, 1, 900))


def test_attention_workspace_is_shared_by_calls_of_any_size():
    """One workspace, garbage behind its counters, calls of different shapes one after another: each as on its own."""
    rng = np.random.default_rng(12)
    shapes = [([5000], [1], 2, 4, 128, 0), ([900, 40, 2500], [1, 1, 1], 1, 8, 64, 0), ([3000, 700], [9, 40], 2, 4, 128, 0),
              ([6000], [1], 1, 2, 256, 1500), ([2000, 2100], [3, 1], 1, 5, 96, 0)]
    cases = []
    for lens, new, heads, group, dim, window in shapes:
        cache, _, _ = random_cache(rng, lens, 64, heads, dim)
        q_start = dev(np.concatenate(([0], np.cumsum(new))).astype(np.int32))
        q = torch.randn(sum(new), heads * group, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(len(cases)))
        cases.append((cache, q, q_start, dev(np.array(lens, np.int32)), max(new), max(lens), window))
    alone = [Z.attn_q4_0(c, q, s, n, a, b, window=w) for c, q, s, n, a, b, w in cases]
    size = max(Z.attn_q4_0_workspace_bytes(c, q.shape[1], a, b) for c, q, s, n, a, b, w in cases)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    ws[:8192] = 0
    for _ in range(2):
        for (c, q, s, n, a, b, w), want in zip(cases, alone):
            assert torch.equal(Z.attn_q4_0(c, q, s, n, a, b, window=w, workspace=ws), want)
    assert not ws[:8192].any()


def test_caches_past_four_gigabytes():
    page, heads, dim = 1024, 4, 256
    per = Z.kv_page_bytes(page, heads, dim)
    n_pages = (9 << 29) // per                              # 4.5 GiB
    pages = torch.zeros(n_pages * per, dtype=torch.uint8, device="cuda")
    cache = Z.KVCache(pages, page, heads, dim, torch.tensor([[n_pages - 1, n_pages - 2]], dtype=torch.int32, device="cuda"))
    g = torch.Generator("cuda").manual_seed(1)
    n = 1100
    k, v = (torch.randn(n, heads, dim, device="cuda", generator=g) for _ in range(2))
    kval, vval = (torch.empty(n, heads, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    Z.kv_append_q4_0(cache, k, v, torch.zeros(n, dtype=torch.int32, device="cuda"),
                     torch.arange(n, dtype=torch.int32, device="cuda"), k_val=kval, v_val=vval)
    assert not pages[:(n_pages - 2) * per].any()
    tail = pages[(n_pages - 2) * per:].cpu().numpy()
    kk, vv = R.values(tail, page, heads, dim)
    for val, have in ((kval, kk), (vval, vv)):
        have = np.concatenate((have[1], have[0]), 1)[:, :n].transpose(1, 0, 2)
        assert np.array_equal(val.cpu().numpy(), have.astype(np.float16))
    q = torch.randn(1, heads, dim, device="cuda", generator=g)
    out = Z.attn_q4_0(cache, q, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                      torch.tensor([n], dtype=torch.int32, device="cuda"), 1, n)
    check_attention(out, q.cpu().numpy(), [0, 1], [n], np.array([[1, 0]]), tail, page, heads, dim)
    del pages, cache
    torch.cuda.empty_cache()
