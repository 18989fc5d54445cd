"""Attention of drafted trees over the cache on the GPU against its formula in 64 bits (tests/tree_ref.py).

Bounds: the result's are those of tests/test_block_ops_gpu.py (the arithmetic is the same). lse: a score is off by at most
2^-19 P as there, the sum of p by 2^-17 of itself, and lse itself takes four fp32 operations on numbers below
|lse| + 16 (in powers of two: 1.45 times that), each off by half a unit, 2^-24 of its result.
"""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests import tree_ref as T
from tests.test_block_ops_gpu import dev, random_cache, ragged

pytestmark = pytest.mark.gpu


def check(out, lse, q, q_start, lens, table, pages, page, heads, dim, masks, window=0, scale=None, rows=None):
    scale = dim ** -0.5 if scale is None else scale
    k, v = R.values(pages, page, heads, dim)
    want, want_lse, tp, tv = T.attention(q, q_start, lens, table, k, v, page, scale, masks, window)
    rows = np.arange(len(q)) if rows is None else rows
    got = out.double().cpu().numpy()[rows]
    want, want_lse, tp, tv = (x[rows] for x in (want, want_lse, tp, tv))
    assert np.isfinite(got).all()
    over = np.abs(got - want) - tv * (2 * 2.0 ** -19 * tp + 2.0 ** -17)[..., None]
    assert (over <= 0).all(), (over.max(), np.abs(got - want).max())
    if lse is None:
        return
    got = lse.double().cpu().numpy()[rows]
    none = np.isneginf(want_lse)
    assert np.array_equal(np.isneginf(got), none) and not np.isnan(got).any()
    w = np.where(none, 0, want_lse)
    over = np.abs(np.where(none, 0, got) - w) - (2.0 ** -19 * tp + 2.0 ** -17 + 8 * 2.0 ** -24 * (np.abs(w) + 16))
    assert (over <= 0).all(), over.max()


def run(rng, lens, new, page, heads, group, dim, masks="tree", window=0, scale=None, words=None, dead=None, sharp=1.5):
    cache, pages, table = random_cache(rng, lens, page, heads, dim, dead=dead)
    q_start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = (sharp * rng.standard_normal((q_start[-1], heads * group, dim))).astype(np.float32)
    if masks == "tree":
        masks = [T.tree_mask(n, rng) for n in new]
    elif masks == "any":
        masks = [rng.random((n, n)) < 0.4 for n in new]
    words = -(-max(new) // 32) if words is None else words
    seen = None if masks is None else dev(T.pack(masks, words))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = torch.full(q.shape, float("nan"), device="cuda"), torch.full(q.shape[:2], float("nan"), device="cuda")
    Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), max(new), max(lens), seen=seen, lse=lse,
                     scale=scale, window=window, out=out, status=status)
    assert status.item() == 0
    check(out, lse, q, q_start, lens, table, pages, page, heads, dim, masks, window, scale)
    return cache, pages, table, q, q_start, masks, seen, out, lse


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads, group, new", [(2, 1, 3), (1, 1, 8), (2, 4, 4), (1, 4, 7), (2, 3, 13), (1, 8, 17)])
def test_tree(dim, heads, group, new):
    """4, 8, 16, 28, 39 and 136 columns; lengths around a tile's and a page's ends."""
    rng = np.random.default_rng(dim + heads + new)
    run(rng, [new, new + 1, 40, 300, 1029], [new, max(1, new - 1), new, 2, new], 32, heads, group, dim)


@pytest.mark.parametrize("masks", ["tree", "any", None])
@pytest.mark.parametrize("lens, new, window", [
    ([5], [5], 0), ([700, 33, 8], [8, 3, 8], 0), ([700, 33, 8], [2, 7, 1], 16), ([1000, 129], [4, 4], 100), ([1000, 129], [4, 4], 1),
    ([600, 50], [70, 50], 0), ([1500], [130], 33), ([90, 1111, 64], [0, 65, 64], 0), ([333], [333], 0), ([400, 47], [33, 31], 40)])
@pytest.mark.parametrize("heads, group, dim", [(2, 4, 128), (3, 1, 64), (1, 7, 256)])
def test_orders(masks, lens, new, window, heads, group, dim):
    """Trees, any bits (rows without one among them, later tokens too), and the ordinary order with lse alone; windows that
    end among the new tokens, more words than the tokens need."""
    run(np.random.default_rng(sum(lens) + sum(new) + window), lens, new, 32, heads, group, dim, masks=masks, window=window,
        words=None if window else 12)


@pytest.mark.parametrize("heads, group, dim, n", [(1, 1, 128, 3), (1, 2, 64, 6), (1, 4, 96, 4), (2, 4, 128, 9), (1, 4, 256, 9)])
def test_rows_that_see_nothing(heads, group, dim, n):
    """No token before the new ones and no bit set: zeros and -infinity, in a call with rows that see something; and more
    new tokens than the cache holds, whose first ones are no tokens of it."""
    rng = np.random.default_rng(n + dim)
    lens, new = [n, 50, 2, 0], [n, n, n, n]
    masks = [rng.random((n, n)) < 0.5 for _ in new]
    masks[0][1] = False
    masks[0][n - 1] = False
    _, _, _, _, q_start, _, _, out, lse = run(rng, lens, new, 16, heads, group, dim, masks=masks)
    for row in (1, n - 1):
        assert not out[row].any() and torch.isneginf(lse[row]).all()
    assert not out[q_start[3]:].any() and torch.isneginf(lse[q_start[3]:]).all()


@pytest.mark.parametrize("heads, group, dim, n", [(1, 1, 128, 4), (1, 2, 128, 4), (1, 4, 128, 4), (2, 4, 128, 12), (2, 4, 64, 40),
                                                  (1, 4, 256, 12), (1, 8, 192, 12)])
@pytest.mark.parametrize("what", ["v", "k"])
def test_unseen_tokens_may_hold_anything(heads, group, dim, n, what):
    """Infinities and NaN in drafted tokens: rows that see no such token are untouched."""
    rng = np.random.default_rng(n * dim + heads)
    page, lens = 32, [n + 37]
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    masks = [T.tree_mask(n, rng)]
    masks[0][:, n // 2] = False
    masks[0][:, n - 1] = False
    masks[0][n - 1, n - 1] = masks[0][n // 2, n // 2] = True
    for j, worst in ((n // 2, np.inf), (n - 1, np.nan)):
        at = lens[0] - n + j
        for h in range(heads):
            R.put(pages, page, heads, dim, table[0, at // page], at % page, h, 1 if what == "v" else 0,
                  np.full(dim, 15), np.full(dim // 32, worst, np.float16))
    cache = Z.KVCache(dev(pages), page, heads, dim, dev(table))
    q = rng.standard_normal((n, heads * group, dim)).astype(np.float32)
    q_start = np.array([0, n], np.int32)
    lse = torch.empty(n, heads * group, device="cuda")
    out = Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), n, lens[0], seen=dev(T.pack(masks, 2)), lse=lse)
    rows = np.array([i for i in range(n) if i not in (n // 2, n - 1)])
    with np.errstate(invalid="ignore"):
        check(out, lse, q, q_start, lens, table, pages, page, heads, dim, masks, rows=rows)


@pytest.mark.parametrize("n_seq, most, new, heads, group, dim, window", [
    (40, 4000, 4, 8, 1, 128, 0), (40, 4000, 2, 8, 4, 128, 900), (60, 2500, 5, 4, 3, 96, 0), (28, 3500, 2, 6, 7, 256, 0)])
def test_many_long_sequences(n_seq, most, new, heads, group, dim, window):
    """Stretches of all sequences' steps a CTA, some sequences without a drafted token; the same bits again."""
    rng = np.random.default_rng(n_seq + most)
    lens = ragged(rng, n_seq, most)
    counts = [int(min(n, rng.integers(0, new + 1))) for n in lens]
    counts[int(np.argmax(lens))] = new
    cache, _, _, q, q_start, _, seen, out, lse = run(rng, lens, counts, 64, heads, group, dim, window=window)
    for _ in range(2):
        again = torch.empty_like(lse)
        o = Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), new, most, seen=seen, lse=again, window=window)
        assert torch.equal(o, out) and torch.equal(again, lse)


@pytest.mark.parametrize("group, n", [(1, 3), (2, 8), (4, 9)])
def test_long_context(group, n):
    """Many parts that are joined, lse among them."""
    rng = np.random.default_rng(group)
    run(rng, [9000], [n], 64, 2, group, 128)


def test_huge_scores():
    """Scores past 2^23: the rows done once more on the form for many columns, with their bits."""
    rng = np.random.default_rng(3)
    for group, n in ((1, 4), (4, 9)):
        cache, pages, table = random_cache(rng, [60], 32, 1, 128)
        q = (3e7 * rng.standard_normal((n, group, 128))).astype(np.float32)
        masks, q_start = [T.tree_mask(n, rng)], np.array([0, n], np.int32)
        lse = torch.empty(n, group, device="cuda")
        out = Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array([60], np.int32)), n, 60, seen=dev(T.pack(masks, 1)), lse=lse)
        k, v = R.values(pages, 32, 1, 128)
        want, want_lse, tp, _ = T.attention(q, q_start, [60], table, k, v, 32, 128 ** -0.5, masks)
        # the largest score stands alone, unless another is within the scores' error
        assert np.isfinite(out.cpu().numpy()).all()
        assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 2.0 ** -19 * tp + 8 * 2.0 ** -24 * np.abs(want_lse) + 1)
        score = np.full((n, group, 60), -np.inf)
        for i in range(n):
            t = T.visible(60, n, i, masks[0])
            kk = k[table[0][np.arange(60) // 32], 0, np.arange(60) % 32]
            score[i][:, t] = (q[i].astype(np.float64) @ kk[t].T) * 128 ** -0.5
        top2 = np.sort(score, -1)[..., -2:]
        clear = top2[..., 1] - top2[..., 0] > 4 * 2.0 ** -19 * tp + 100
        assert clear.mean() > 0.8
        at = table[0][score.argmax(-1) // 32], score.argmax(-1) % 32
        best = v[at[0], 0, at[1]]
        err = np.abs(out.double().cpu().numpy() - best)[clear]
        assert np.all(err <= 2.0 ** -17 * np.abs(best[clear]).reshape(-1, 4, 32).max(-1).repeat(32, -1))


def test_bad_sequences():
    rng = np.random.default_rng(4)
    cache, pages, table = random_cache(rng, [40, 50, 60], 16, 2, 128)
    n = 5
    masks = [T.tree_mask(n, rng) for _ in range(3)]
    q_start = np.arange(0, 16, 5).astype(np.int32)
    q = rng.standard_normal((15, 8, 128)).astype(np.float32)
    for lens in ([40, -1, 60], [40, 61, 60]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        lse = torch.zeros(15, 8, device="cuda")
        out = Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), n, 60, seen=dev(T.pack(masks, 1)), lse=lse,
                               status=status)
        assert status.item() == 1 and out[5:10].isnan().all() and lse[5:10].isnan().all()
        check(out, lse, q, q_start, [40, 50, 60], table, pages, 16, 2, 128, masks, rows=np.r_[0:5, 10:15])
    # a page number out of range
    bad = table.copy()
    bad[2, 1] = 1 << 20
    broken = Z.KVCache(cache.pages, 16, 2, 128, dev(bad))
    status.zero_()
    out = Z.attn_tree_q4_0(broken, dev(q), dev(q_start), dev(np.array([40, 50, 60], np.int32)), n, 60, seen=dev(T.pack(masks, 1)),
                           lse=lse, status=status)
    assert status.item() == 1 and out[10:].isnan().all() and lse[10:].isnan().all()
    check(out, lse, q, q_start, [40, 50, 60], table, pages, 16, 2, 128, masks, rows=np.r_[0:10])
    assert Z.device_status() == 0


def test_streams_and_graphs():
    """A captured call replays with other trees and lengths; calls on two streams with a workspace each."""
    rng = np.random.default_rng(8)
    heads, group, dim, page, n = 2, 4, 128, 32, 6
    cache, pages, table = random_cache(rng, [900, 300], page, heads, dim)
    q_start = np.array([0, n, 2 * n], np.int32)
    q = [rng.standard_normal((2 * n, heads * group, dim)).astype(np.float32) for _ in range(2)]
    masks = [[T.tree_mask(n, rng) for _ in range(2)] for _ in range(2)]
    lens = [[900, 300], [517, 6]]
    qd, sd, ld = dev(q[0]), dev(T.pack(masks[0], 1)), dev(np.array(lens[0], np.int32))
    out, lse = torch.empty(2 * n, heads * group, dim, device="cuda"), torch.empty(2 * n, heads * group, device="cuda")
    starts, ws = dev(q_start), Z.attn_q4_0_workspace(cache, heads * group, n, 900)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda: Z.attn_tree_q4_0(cache, qd, starts, ld, n, 900, seen=sd, lse=lse, out=out, workspace=ws, stream=side)  # noqa: E731
    with torch.cuda.stream(side):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for i in (0, 1, 0):
        torch.cuda.synchronize()
        qd.copy_(dev(q[i]))
        sd.copy_(dev(T.pack(masks[i], 1)))
        ld.copy_(dev(np.array(lens[i], np.int32)))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        check(out, lse, q[i], q_start, lens[i], table, pages, page, heads, dim, masks[i])
    other = torch.cuda.Stream()
    results = []
    for _ in range(4):
        for st in (side, other):
            results.append(Z.attn_tree_q4_0(cache, qd, starts, ld, n, 900, seen=sd, stream=st))
    torch.cuda.synchronize()
    assert all(torch.equal(r, out) for r in results)


# More columns times tiles than 16 columns a CTA are for: heads of up to 128 dimensions on tcgen05.
@pytest.mark.parametrize("dim, heads, group, new, length, window, masks", [
    (128, 8, 4, 16, 9300, 0, "tree"), (64, 16, 4, 24, 12500, 0, "tree"), (96, 8, 4, 33, 9500, 0, "any"), (128, 8, 4, 40, 9100, 6400, "tree"),
    (128, 8, 4, 25, 9200, 0, None)])
def test_many_columns_and_tokens(dim, heads, group, new, length, window, masks):
    rng = np.random.default_rng(dim + new)
    cache, _, _, q, q_start, _, seen, out, lse = run(rng, [length], [new], 64, heads, group, dim, masks=masks, window=window)
    again = torch.empty_like(lse)
    o = Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array([length], np.int32)), new, length, seen=seen, lse=again, window=window)
    assert torch.equal(o, out) and torch.equal(again, lse)


def test_many_columns_and_sequences():
    rng = np.random.default_rng(31)
    lens = [3000, 0, 1, 700, 2999, 25, 1800]
    run(rng, lens, [25, 0, 1, 9, 25, 25, 13], 32, 8, 4, 128)
    run(rng, lens, [25, 3, 2, 9, 25, 25, 13], 16, 8, 4, 96, masks="any", window=900)


@pytest.mark.parametrize("what", ["v", "k", "scores"])
def test_many_columns_with_rows_done_once_more(what):
    """Infinities and NaN in drafted tokens that most rows do not see, and scores past 2^23, on tcgen05 (rows token by token)."""
    rng = np.random.default_rng(5)
    page, heads, group, dim, n, length = 64, 8, 4, 128, 16, 9300
    cache, pages, table = random_cache(rng, [length], page, heads, dim)
    masks = [T.tree_mask(n, rng)]
    masks[0][:, 7] = False
    masks[0][:, 12] = False
    masks[0][7, 7] = masks[0][12, 12] = True
    for j, worst in ((7, np.inf), (12, np.nan)) if what != "scores" else ():
        at = length - n + j
        for h in range(heads):
            R.put(pages, page, heads, dim, table[0, at // page], at % page, h, 1 if what == "v" else 0, np.full(dim, 15),
                  np.full(dim // 32, worst, np.float16))
    cache = Z.KVCache(dev(pages), page, heads, dim, dev(table))
    q = (rng.standard_normal((n, heads * group, dim)) * (3e7 if what == "scores" else 1)).astype(np.float32)
    q_start, lse = np.array([0, n], np.int32), torch.empty(n, heads * group, device="cuda")
    out = Z.attn_tree_q4_0(cache, dev(q), dev(q_start), dev(np.array([length], np.int32)), n, length, seen=dev(T.pack(masks, 1)), lse=lse)
    rows = np.array([i for i in range(n) if i not in (7, 12)])
    if what != "scores":
        with np.errstate(invalid="ignore"):
            check(out, lse, q, q_start, [length], table, pages, page, heads, dim, masks, rows=rows)
        return
    k, v = R.values(pages, page, heads, dim)
    _, want_lse, tp, _ = T.attention(q, q_start, [length], table, k, v, page, dim ** -0.5, masks)
    assert np.isfinite(out.cpu().numpy()).all()
    # ln of at most 9300 equal terms above the largest score
    assert np.all(np.abs(lse.double().cpu().numpy() - want_lse) <= 2.0 ** -19 * tp + 8 * 2.0 ** -24 * np.abs(want_lse) + 10)
