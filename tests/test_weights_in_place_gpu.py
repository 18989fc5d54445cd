"""Sums in place: behind windows (where the kernel for few columns begins at the first tile that a row sees), over more sequences than a
CTA has threads, and on a cache that was cut back. Bounds: tests/test_keep_gpu.py."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests import tree_ref as T
from tests.test_block_ops_gpu import dev, make_cache, ragged
from tests.test_keep_gpu import run_weights

pytestmark = pytest.mark.gpu


def in_place(call, new, lens, masks, window, keep=1.0):
    """The same call with out the sums themselves; and what a window leaves alone."""
    cache, q, starts, ld, lse, had, out = call
    sums = had.clone()
    seen = None if masks is None else dev(T.pack(masks, -(-max(new) // 32)))
    Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, max(new), max(lens), seen=seen, window=window, sums=sums, out=sums, keep=keep)
    for s, n in enumerate(lens):
        assert torch.equal(sums[s, :, :n], out[s, :, :n]) and torch.equal(sums[s, :, n:], had[s, :, n:])
        gone = max(0, n - new[s] - window) if window else 0
        if keep == 1.0:
            assert torch.equal(sums[s, :, :gone], had[s, :, :gone])
    assert Z.device_status() == 0


@pytest.mark.parametrize("window", [1, 15, 16, 17, 40, 64, 100, 300])
@pytest.mark.parametrize("heads, group, dim, new", [(2, 1, 128, 1), (1, 4, 64, 1), (3, 2, 256, 3), (2, 8, 96, 3), (1, 8, 128, 20)])
@pytest.mark.parametrize("tree", [False, True])
def test_windows(window, heads, group, dim, new, tree):
    """First tiles of odd and even number; sequences without rows, shorter than the window, and empty."""
    rng = np.random.default_rng(window + dim)
    lens = [700, 333, 416, 417, 431, 432, 90, 7, 0, 512]
    counts = [min(new, n) for n in lens]
    counts[3] = counts[9] = 0
    masks = [T.tree_mask(n, rng) for n in counts] if tree else None
    in_place(run_weights(rng, lens, counts, 16, heads, group, dim, masks=masks, window=window, wide=3), counts, lens, masks, window)


@pytest.mark.parametrize("n_seq, group, new, keep", [(257, 4, 1, 1.0), (300, 1, 1, 0.5), (600, 4, 2, 1.0), (300, 4, 8, 0.9)])
def test_many_sequences(n_seq, group, new, keep):
    """More sequences than the 256 threads that look for a CTA's stretch, many of them empty or without rows, some long."""
    rng = np.random.default_rng(n_seq)
    lens = [int(n) for n in ragged(rng, n_seq, 120)]
    for s in range(0, n_seq, 7):
        lens[s] = 0
    lens[255], lens[256], lens[n_seq - 1] = 900, 0, 2100
    counts = [min(n, 1 + s % new) if s % 5 else 0 for s, n in enumerate(lens)]
    counts[n_seq - 1] = new
    in_place(run_weights(rng, lens, counts, 32, 2, group, 64, keep=keep, wide=1), counts, lens, None, 0, keep)


def test_sums_on_a_cache_that_was_cut_back():
    """Weights, eviction with the kept sums, and then steps that append trees to the cut cache, add their weights to those sums in place
    and keep a path: the sums against 64 bits at each step."""
    rng = np.random.default_rng(8)
    heads, group, dim, page, budget = 2, 4, 128, 16, 90
    hq, lens = heads * group, [400, 91, 60]
    cache, q, starts, ld, lse, had, out = run_weights(rng, lens, [2, 2, 2], page, heads, group, dim)
    per = 10
    table = rng.permutation(3 * per).reshape(3, per)
    cut, _ = make_cache(3 * per, page, heads, dim, table, fill=0)
    sums, now = torch.zeros(3, heads, per * page, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    index = Z.kv_evict_q4_0(cache, cut, ld, out, budget, max(lens), sinks=2, recent=20, sums_out=sums, len_out=now)
    want = T.evict_index(out.cpu().numpy(), lens, budget, 2, 20)
    assert np.array_equal(index.cpu().numpy(), want)
    kept = np.where(want >= 0, np.take_along_axis(out.cpu().numpy(), np.maximum(want, 0), 2), 0)
    assert np.array_equal(sums.cpu().numpy()[:, :, :budget], kept)
    lens = now.tolist()
    assert lens == [90, 90, 60]
    rope = dev(R.rope_table(600, dim))
    for step, counts in enumerate(([3, 1, 7], [1, 9, 2], [12, 12, 12])):
        n, words = sum(counts), 1
        masks = [T.tree_mask(c, rng) for c in counts]
        first = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
        slots = np.concatenate([lens[s] + np.arange(counts[s]) for s in range(3)]).astype(np.int32)
        turns = (410 + 20 * step + np.concatenate([m.sum(1) for m in masks])).astype(np.int32)
        x = dev(rng.standard_normal((n, hq + 2 * heads, dim)).astype(np.float32))
        qs = Z.kv_append_q4_0(cut, x[:, hq:hq + heads], x[:, hq + heads:], dev(np.repeat(np.arange(3), counts).astype(np.int32)), dev(slots),
                              q=x[:, :hq], rope=rope, rope_pos=dev(turns))
        long = [lens[s] + counts[s] for s in range(3)]
        ld, starts, seen = dev(np.array(long, np.int32)), dev(first), dev(T.pack(masks, words))
        lse, before = torch.empty(n, hq, device="cuda"), sums.cpu().numpy().astype(np.float64)
        Z.attn_tree_q4_0(cut, qs, starts, ld, max(counts), max(long), seen=seen, lse=lse)
        Z.attn_weights_q4_0(cut, qs, starts, ld, lse, max(counts), max(long), seen=seen, sums=sums, out=sums, keep=0.75)
        k, _ = R.values(cut.pages.cpu().numpy(), page, heads, dim)
        add, tol = T.weights(qs.cpu().numpy(), first, long, table, k, page, dim ** -0.5, lse.double().cpu().numpy(), masks)
        got = sums.double().cpu().numpy()
        for s in range(3):
            total = add[s, :, :long[s]].copy()
            total[:, :lens[s]] += 0.75 * before[s, :, :lens[s]]
            assert np.all(np.abs(got[s, :, :long[s]] - total) <= 2.0 ** -18 * tol[s, :, :long[s]] + 2.0 ** -24 * total + 1e-30)
        paths = [np.flatnonzero(m[rng.integers(0, len(m))]) for m in masks]
        path = np.zeros((3, max(map(len, paths))), np.int32)
        for s, p in enumerate(paths):
            path[s, :len(p)] = p
        new = Z.kv_accept_q4_0(cut, dev(np.array(lens, np.int32)), dev(path), dev(np.array([len(p) for p in paths], np.int32)), sums=sums)
        after = sums.double().cpu().numpy()
        for s, p in enumerate(paths):
            got[s, :, lens[s]:lens[s] + len(p)] = got[s][:, lens[s] + p]
            lens[s] += len(p)
            assert np.array_equal(after[s, :, :lens[s]], got[s, :, :lens[s]])
        assert new.tolist() == lens
    assert Z.device_status() == 0
