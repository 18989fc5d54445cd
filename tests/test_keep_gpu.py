"""What stays in the cache, on the GPU: the weights that attention gives its tokens, eviction by them, the accepted path of a
drafted tree, and the append whose rotation has positions of its own.

Bounds: eviction, acceptance and the append move bytes and pick whole numbers: equal. A token's weight is a sum of p = exp(score
- lse): a score is off by at most 2^-19 P, P = scale sum |q_e| max|k_block| (tests/test_block_ops_gpu.py), p's relative error
is twice that, the fma of p's exponent and the product of lse add 2^-23 (P + |lse|), the exponential 2^-21, and at most 1024 / 4
additions in a row 2^-16 of the sum: together below 2^-18 (P + |lse| + 16) a term.
"""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests import tree_ref as T
from tests.test_block_ops_gpu import dev, make_cache, random_cache, ragged

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weights
def run_weights(rng, lens, new, page, heads, group, dim, masks=None, window=0, keep=1.0, before=True, sharp=1.5, wide=0):
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    q_start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = (sharp * rng.standard_normal((q_start[-1], heads * group, dim))).astype(np.float32)
    if masks == "tree":
        masks = [T.tree_mask(n, rng) for n in new]
    seen = None if masks is None else dev(T.pack(masks, -(-max(new) // 32)))
    starts, ld, most = dev(q_start), dev(np.array(lens, np.int32)), max(lens)
    lse = torch.empty(q.shape[:2], device="cuda")
    Z.attn_tree_q4_0(cache, dev(q), starts, ld, max(new), most, seen=seen, lse=lse, window=window)
    old = np.abs(rng.standard_normal((len(lens), heads, most + wide))).astype(np.float32)
    had = dev(old) if before else None
    out = torch.full(old.shape, -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, max(new), most, seen=seen, window=window, sums=had, out=out, keep=keep,
                        status=status)
    assert status.item() == 0 and Z.device_status() == 0
    k, _ = R.values(pages, page, heads, dim)
    want, tol = T.weights(q, q_start, lens, table, k, page, dim ** -0.5, lse.double().cpu().numpy(), masks, window)
    got = out.double().cpu().numpy()
    for s, n in enumerate(lens):
        add, bound = want[s, :, :n].copy(), 2.0 ** -18 * tol[s, :, :n] + 1e-30
        rest = n - new[s]
        if before and rest > 0:
            add[:, :rest] += float(np.float32(keep)) * old[s, :, :rest].astype(np.float64)
            bound = bound + 2.0 ** -24 * np.abs(add)
        over = np.abs(got[s, :, :n] - add) - bound
        assert n == 0 or (over <= 0).all(), (s, over.max(), np.unravel_index(over.argmax(), over.shape))
        assert np.all(got[s, :, n:] == -7.0)
    return cache, q, starts, ld, lse, had, out


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads, group", [(1, 1), (2, 4), (1, 8), (2, 5), (1, 24)])
def test_weights_one_token(dim, heads, group):
    run_weights(np.random.default_rng(dim + heads), [1, 16, 37, 300, 1029, 0], [1] * 6, 32, heads, group, dim)


@pytest.mark.parametrize("masks", [None, "tree"])
@pytest.mark.parametrize("lens, new, window, keep, before", [
    ([700, 33, 8], [8, 3, 8], 0, 1.0, True), ([700, 33, 8], [2, 7, 1], 16, 0.5, True), ([1000, 129], [4, 4], 1, 0.0, True),
    ([600, 50, 3], [70, 50, 0], 0, 1.0, False), ([1500], [130], 33, 0.9, True), ([333], [333], 0, 1.0, True),
    ([3, 40, 0], [6, 2, 2], 0, 1.0, True)])
@pytest.mark.parametrize("heads, group, dim", [(2, 4, 128), (3, 1, 64), (1, 7, 256)])
def test_weights_new_tokens(masks, lens, new, window, keep, before, heads, group, dim):
    """Several new tokens, up to fifteen blocks of columns (keep is a C float); windows, trees, rows that see nothing, sequences without a row."""
    run_weights(np.random.default_rng(sum(lens) + window), lens, new, 16, heads, group, dim, masks=masks, window=window, keep=keep,
                before=before, wide=5)


def test_weights_of_a_row_add_up_to_one():
    rng = np.random.default_rng(2)
    cache, q, starts, ld, lse, _, out = run_weights(rng, [5000, 2500], [1, 1], 64, 4, 2, 128, before=False, wide=3)
    w = out.double()
    w[:, :, 5000:] = 0
    w[1, :, 2500:] = 0
    # 2 rows of a kv head; the weights' own errors: 2^-18 (P + |lse| + 16) with P below 500 here
    assert (w.sum(-1) - 2).abs().max() < 2 * 2.0 ** -18 * 530


def test_weights_in_place_and_again():
    rng = np.random.default_rng(3)
    lens = ragged(rng, 40, 3000)
    new = [1 if n else 0 for n in lens]
    cache, q, starts, ld, lse, had, out = run_weights(rng, lens, new, 16, 4, 4, 128)
    most = max(lens)
    again = torch.full_like(out, -7.0)
    Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, 1, most, sums=had, out=again)
    assert torch.equal(again, out)
    in_place = had.clone()
    Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, 1, most, sums=in_place, out=in_place)
    for s, n in enumerate(lens):
        assert torch.equal(in_place[s, :, :n], out[s, :, :n]) and torch.equal(in_place[s, :, n:], had[s, :, n:])
    # without rows: what stood there, times keep
    half = torch.full_like(out, -7.0)
    none = torch.zeros(41, dtype=torch.int32, device="cuda")
    Z.attn_weights_q4_0(cache, torch.empty(0, 16, 128, device="cuda"), none, ld, torch.empty(0, 16, device="cuda"), 1, most, sums=had,
                        out=half, keep=0.5)
    for s, n in enumerate(lens):
        assert torch.equal(half[s, :, :n], 0.5 * had[s, :, :n])


@pytest.mark.parametrize("group, new", [(4, 1), (4, 6), (8, 20)])
def test_weights_of_unseen_tokens(group, new):
    """Infinities and NaN in keys that a row does not see give nobody anything but those who see them."""
    rng = np.random.default_rng(group + new)
    page, dim, n = 32, 128, 200
    cache, pages, table = random_cache(rng, [n], page, 1, dim)
    masks = [np.tril(np.ones((new, new), bool))]
    masks[0][:, new // 2] = False
    window = 64
    for at, worst in ((3, np.nan), (40, np.inf), (n - new + new // 2, np.nan)):
        R.put(pages, page, 1, dim, table[0, at // page], at % page, 0, 0, np.full(dim, 15), np.full(dim // 32, worst, np.float16))
    cache = Z.KVCache(dev(pages), page, 1, dim, dev(table))
    q = rng.standard_normal((new, group, dim)).astype(np.float32)
    starts, ld = dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32))
    lse, seen = torch.empty(new, group, device="cuda"), dev(T.pack(masks, 1))
    Z.attn_tree_q4_0(cache, dev(q), starts, ld, new, n, seen=seen, lse=lse, window=window)
    assert torch.isfinite(lse).all()
    out = Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, new, n, seen=seen, window=window)
    assert torch.isfinite(out).all() and not out[0, 0, [3, 40, n - new + new // 2]].any()
    assert abs(out.double().sum().item() - new * group) < new * group * 2.0 ** -18 * 128  # P + |lse| + 16 is below 128 here


def test_weights_bad_sequences_and_pages():
    rng = np.random.default_rng(5)
    lens = [40, 50, 60]
    cache, pages, table = random_cache(rng, lens, 16, 2, 128)
    starts, q = dev(np.arange(4).astype(np.int32)), dev(rng.standard_normal((3, 8, 128)).astype(np.float32))
    lse = torch.empty(3, 8, device="cuda")
    good = dev(np.array(lens, np.int32))
    Z.attn_tree_q4_0(cache, q, starts, good, 1, 60, lse=lse)
    want = Z.attn_weights_q4_0(cache, q, starts, good, lse, 1, 60)
    for n in (-3, 61):
        status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((3, 2, 60), -7.0, device="cuda")
        Z.attn_weights_q4_0(cache, q, starts, dev(np.array([40, n, 60], np.int32)), lse, 1, 60, out=out, status=status)
        assert status.item() == 1 and torch.all(out[1] == -7) and torch.equal(out[0, :, :40], want[0, :, :40]) and torch.equal(out[2], want[2])
    table[2, 1] = -1
    broken = Z.KVCache(cache.pages, 16, 2, 128, dev(table))
    status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((3, 2, 60), -7.0, device="cuda")
    Z.attn_weights_q4_0(broken, q, starts, good, lse, 1, 60, out=out, status=status)
    assert status.item() == 1 and torch.all(out[2, :, 16:32] == -7)
    assert torch.equal(out[2, :, :16], want[2, :, :16]) and torch.equal(out[2, :, 32:], want[2, :, 32:])
    assert Z.device_status() == 0


@pytest.mark.parametrize("group, new", [(4, 1), (4, 3), (8, 20)])
def test_pages_before_the_window_may_be_gone(group, new):
    """A windowed sequence's first pages have no number any more: neither the attention nor the weights look at them (the first
    page is in a tile of 128 tokens with some that are seen), and their tokens' sums are kept."""
    rng = np.random.default_rng(new)
    page, dim, n, window = 16, 128, 700, 230
    cache, pages, table = random_cache(rng, [n], page, 1, dim)
    masks = [T.tree_mask(new, rng)]
    q, starts, ld = dev(rng.standard_normal((new, group, dim)).astype(np.float32)), dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32))
    seen, had = dev(T.pack(masks, 1)), torch.rand(1, 1, n, device="cuda")
    gone = table.copy()
    gone[0, :(n - new - window) // page] = -1
    results = []
    for t in (table, gone):
        c, lse, status = Z.KVCache(cache.pages, page, 1, dim, dev(t)), torch.empty(new, group, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        out = Z.attn_tree_q4_0(c, q, starts, ld, new, n, seen=seen, lse=lse, window=window, status=status)
        w = Z.attn_weights_q4_0(c, q, starts, ld, lse, new, n, seen=seen, window=window, sums=had, keep=0.5, status=status)
        assert status.item() == 0
        results.append((out, lse, w))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert torch.equal(w[0, 0, :n - new - window], 0.5 * had[0, 0, :n - new - window])


# ------------------------------------------------------------------ eviction
def gathered(pages, page, heads, dim, table, index, to_pages, to_page, to_table):
    """The bytes of `to` after the move, by plain numpy."""
    codes = R.unpack(pages, page, heads, dim)
    want = to_pages.copy()
    for s in range(index.shape[0]):
        n = int((index[s, 0] >= 0).sum())
        for tile in range(-(-n // 16)):
            t = want.reshape(-1, heads, to_page // 16, 18 * dim)[to_table[s, tile * 16 // to_page], :, tile % (to_page // 16)]
            t[:] = 0
        for h in range(heads):
            for j in range(-(-n // 16) * 16):
                where = to_table[s, j // to_page], j % to_page, h
                if j >= n:
                    for which in (0, 1):
                        R.put(want, to_page, heads, dim, *where, which, np.zeros(dim, int), np.zeros(dim // 32, np.float16))
                    continue
                src = table[s, index[s, h, j] // page], h, index[s, h, j] % page
                for which in (0, 1):
                    R.put(want, to_page, heads, dim, *where, which, codes[which][src] + 8, codes[2 + which][src])
    return want


def some_sums(rng, shape, kind):
    x = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "ties":
        x = np.where(rng.random(shape) < 0.7, rng.choice(np.array([0.0, -0.0, 1.0, 2.0], np.float32), shape), x)
    elif kind == "equal":
        x[:] = 0.25
    elif kind == "any":
        x = rng.choice(np.array([np.nan, np.inf, -np.inf, -1.5, 0.0, -0.0, 1e-42, -1e-42, 3.4e38], np.float32), shape)
    return x


def run_evict(rng, lens, budget, sinks, recent, page, to_page, heads, dim, kind="spread", moved=True, wide=0):
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    most = max(lens)
    sums = some_sums(rng, (len(lens), heads, most + wide), kind)
    per = -(-budget // to_page)
    to_table = rng.permutation(len(lens) * per).reshape(len(lens), per)
    to, to_pages = make_cache(len(lens) * per, to_page, heads, dim, to_table, seed=3)
    out = torch.full((len(lens), heads, budget + wide), -7.0, device="cuda")
    new, status = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    index = Z.kv_evict_q4_0(cache, to, dev(np.array(lens, np.int32)), dev(sums), budget, most, sinks=sinks, recent=recent, sums_out=out,
                            len_out=new, status=status)
    want = T.evict_index(sums, lens, budget, sinks, recent)
    assert np.array_equal(index.cpu().numpy(), want) and status.item() == 0
    assert new.tolist() == [min(n, budget) for n in lens]
    kept = np.where(want >= 0, np.take_along_axis(sums, np.maximum(want, 0), 2), np.float32(0))
    got = out.cpu().numpy()
    assert np.array_equal(got[..., :budget].view(np.uint32), kept.astype(np.float32).view(np.uint32)) and np.all(got[..., budget:] == -7)
    if moved:
        assert np.array_equal(to.pages.cpu().numpy(), gathered(pages, page, heads, dim, table, want, to_pages, to_page, to_table))
    assert np.array_equal(cache.pages.cpu().numpy(), pages)
    return cache, to, sums, index


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page, to_page", [(16, 16), (48, 32), (32, 128)])
def test_evict(dim, page, to_page):
    run_evict(np.random.default_rng(dim + page), [200, 90, 91, 1, 0], 90, 4, 17, page, to_page, 2, dim, wide=3)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "any"])
@pytest.mark.parametrize("lens, budget, sinks, recent", [
    ([33], 32, 0, 0), ([1000, 7, 64], 64, 0, 64), ([1000, 7, 64], 64, 64, 0), ([513, 512, 511], 1, 0, 0), ([3000, 2500], 2400, 3, 100),
    ([600], 599, 1, 1), ([17, 18], 16, 15, 1)])
def test_evict_picks(kind, lens, budget, sinks, recent):
    run_evict(np.random.default_rng(sum(lens) + budget), lens, budget, sinks, recent, 64, 64, 3, 64, kind=kind, moved=False)


@pytest.mark.parametrize("kind", ["spread", "ties", "equal"])
@pytest.mark.parametrize("lens, budget", [([8193, 8192, 100], 4000), ([20481, 20480], 9000), ([50001], 1500), ([70001, 33333], 16000), ([180000, 9], 2000),
                                          ([300007], 150001), ([420003], 1017)])
def test_evict_long(kind, lens, budget):
    """Clusters of CTAs a kv head; sums past what their shared memory holds."""
    run_evict(np.random.default_rng(budget), lens, budget, 16, 1000, 1024, 1024, 1, 64, kind=kind, moved=False)


def test_evict_long_moves():
    run_evict(np.random.default_rng(9), [9000, 2000], 700, 4, 300, 64, 128, 1, 64)


def test_evict_bad_sequences_and_pages():
    rng = np.random.default_rng(6)
    lens, heads, dim, page = [100, 120, 140], 2, 128, 16
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    sums = dev(some_sums(rng, (3, heads, 140), "spread"))
    to_table = np.arange(12).reshape(3, 4)
    fresh = lambda: make_cache(12, page, heads, dim, to_table, seed=4)  # noqa: E731
    to, before = fresh()
    want = Z.kv_evict_q4_0(cache, to, dev(np.array(lens, np.int32)), sums, 64, 140)
    good = to.pages.clone()
    for n in (-1, 141, 1 << 20):
        to, _ = fresh()
        status, new = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
        out = torch.full((3, heads, 64), -7.0, device="cuda")
        index = Z.kv_evict_q4_0(cache, to, dev(np.array([100, n, 140], np.int32)), sums, 64, 140, sums_out=out, len_out=new, status=status)
        assert status.item() == 1 and new.tolist() == [64, -1, 64] and torch.all(index[1] == -1) and not out[1].any()
        assert torch.equal(index[0], want[0]) and torch.equal(index[2], want[2])
        assert torch.equal(to.pages.view(3, -1)[::2], good.view(3, -1)[::2])
        assert np.array_equal(to.pages.view(3, -1)[1].cpu().numpy(), before.reshape(3, -1)[1])
    # a bad page of `from`: its tokens are NaN; one of `to`: not written
    broken = table.copy()
    broken[0, 2] = 1 << 20
    to, _ = fresh()
    status.zero_()
    index = Z.kv_evict_q4_0(Z.KVCache(cache.pages, page, heads, dim, dev(broken)), to, dev(np.array(lens, np.int32)), sums, 64, 140,
                            status=status)
    assert status.item() == 1 and torch.equal(index, want)
    k, v = R.values(to.pages.cpu().numpy(), page, heads, dim)
    for h in range(heads):
        lost = (want[0, h].cpu().numpy() // page == 2)[:64]
        assert lost.any() and np.array_equal(np.isnan(k[:4, h].reshape(64, dim)).all(1), lost)
        assert np.array_equal(np.isnan(v[:4, h].reshape(64, dim)).any(1), lost)
    bad_to = to_table.astype(np.int32)
    bad_to[1, 3] = -5
    to = Z.KVCache(dev(before), page, heads, dim, dev(bad_to))
    status.zero_()
    Z.kv_evict_q4_0(cache, to, dev(np.array(lens, np.int32)), sums, 64, 140, status=status)
    now = to.pages.view(12, -1)
    assert status.item() == 1 and torch.equal(now[:7], good.view(12, -1)[:7]) and torch.equal(now[8:], good.view(12, -1)[8:])
    assert np.array_equal(now[7].cpu().numpy(), before.reshape(12, -1)[7])
    assert Z.device_status() == 0


# ------------------------------------------------------------------ the accepted path
@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("page", [16, 48])
def test_accept(dim, page):
    rng = np.random.default_rng(dim + page)
    heads, paths = 3, [[0, 2, 3, 7], [], [1], [5, 6, 9], list(range(0, 80, 2)), [0, 1, 2], sorted(rng.choice(90, 60, replace=False).tolist())]
    base = [0, 30, 15, 100, 7, 16, 33]
    lens = [b + 95 for b in base]
    cache, pages, table = random_cache(rng, lens, page, heads, dim, dead=0x5A)
    most = max(map(len, paths))
    path = np.full((len(base), most), -3, np.int32)
    for s, p in enumerate(paths):
        path[s, :len(p)] = p
    new, status = torch.empty(len(base), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    old_sums = rng.standard_normal((len(base), heads, max(lens))).astype(np.float32)
    sums = dev(old_sums)
    Z.kv_accept_q4_0(cache, dev(np.array(base, np.int32)), dev(path), dev(np.array([len(p) for p in paths], np.int32)), sums=sums,
                     len_out=new, status=status)
    codes = R.unpack(pages, page, heads, dim)
    want = pages.copy()
    for s, p in enumerate(paths):
        for j, i in enumerate(p):
            for h in range(heads):
                src = table[s, (base[s] + i) // page], h, (base[s] + i) % page
                for which in (0, 1):
                    R.put(want, page, heads, dim, table[s, (base[s] + j) // page], (base[s] + j) % page, h, which, codes[which][src] + 8,
                          codes[2 + which][src])
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    assert new.tolist() == [b + len(p) for b, p in zip(base, paths)] and status.item() == 0
    want_sums = old_sums.copy()
    for s, p in enumerate(paths):
        want_sums[s][:, base[s]:base[s] + len(p)] = old_sums[s][:, base[s] + np.array(p, int)]
    assert np.array_equal(sums.cpu().numpy(), want_sums)


def test_accept_the_longest_path():
    rng = np.random.default_rng(1)
    n, page, heads, dim = 2048, 64, 1, 64
    cache, pages, table = random_cache(rng, [n + 5], page, heads, dim)
    path = np.arange(1, n, 2, dtype=np.int32)
    Z.kv_accept_q4_0(cache, dev(np.array([5], np.int32)), dev(path[None]), dev(np.array([1024], np.int32)))
    old, new = (np.concatenate([x.transpose(0, 2, 1, 3)[table[0, :-1]].reshape(-1, x.shape[-1]) for x in R.unpack(p, page, heads, dim)], 1)
                for p in (pages, cache.pages.cpu().numpy()))
    assert np.array_equal(new[:n + 5][5:5 + 1024], old[5 + path]) and np.array_equal(new[:5], old[:5]) and np.array_equal(new[1029:n + 5], old[1029:n + 5])


def test_accept_bad_sequences():
    rng = np.random.default_rng(2)
    page, heads, dim = 16, 2, 128
    cache, pages, table = random_cache(rng, [64] * 9, page, heads, dim, spare=0)
    table[7, 2] = 99
    cache = Z.KVCache(cache.pages, page, heads, dim, dev(table))
    base = np.array([-1, 10, 10, 10, 10, 10, 60, 30, 20], np.int32)
    path = np.array([[0, 2, 3], [2, 2, 3], [-1, 2, 3], [3, 2, 4], [0, 1, 2], [0, 1, 2], [1, 2, 4], [1, 2, 5], [1, 2, 5]], np.int32)
    count = np.array([3, 3, 3, 3, 4, -1, 3, 3, 3], np.int32)
    new, status = torch.empty(9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    Z.kv_accept_q4_0(cache, dev(base), dev(path), dev(count), len_out=new, status=status)
    assert status.item() == 1 and new.tolist() == [-1] * 8 + [23]
    now = cache.pages.cpu().numpy().reshape(-1, len(pages) // (len(pages) // Z.kv_page_bytes(page, heads, dim)))
    old = pages.reshape(now.shape)
    touched = np.flatnonzero((now != old).any(1))
    assert set(touched) <= set(table[8].tolist()) and len(touched) > 0


# ------------------------------------------------------------------ append with positions of its own
@pytest.mark.parametrize("dim, rot, halves", [(64, 34, False), (96, 96, True), (128, 128, True), (256, 64, False), (128, 0, True)])
@pytest.mark.parametrize("n", [9, 1500])
def test_append_at(dim, rot, halves, n):
    """A token's slot and its rotation's position differ: the same bytes and queries as an append at the rotation's position,
    elsewhere; both kernels."""
    rng = np.random.default_rng(dim + n)
    page, heads, group = 32, 4, 2
    seq, slot = (np.arange(n) % 2).astype(np.int32), (np.arange(n) // 2).astype(np.int32)
    turn = rng.integers(0, 4000, n).astype(np.int32)
    slot[n // 2] = -1
    turn[n // 2] = -1
    per = -(-n // page) + 1
    table = rng.permutation(2 * per).reshape(2, per)
    cache, pages = make_cache(2 * per, page, heads, dim, table)
    x = rng.standard_normal((n, heads * (group + 2), dim)).astype(np.float32)
    q, k, v = (dev(t) for t in np.split(x, [heads * group, heads * (group + 1)], 1))
    rope = None if rot == 0 else dev(R.rope_table(4000, rot))
    kv = [torch.empty(n, heads, dim, dtype=torch.float16, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Z.kv_append_q4_0(cache, k, v, dev(seq), dev(slot), q=q, rope=rope, rope_style=Z.ROPE_HALVES if halves else Z.ROPE_PAIRS,
                           k_val=kv[0], v_val=kv[1], status=status, rope_pos=dev(turn))
    assert status.item() == 0
    live = slot >= 0
    turned = x[:, :heads * (group + 1)].copy()
    if rot:
        turned[live] = R.rotate(turned[live], rope.cpu().numpy(), turn[live], halves)
    assert np.array_equal(out.cpu().numpy(), np.where(live[:, None, None], turned[:, :heads * group], 0))
    got = R.unpack(cache.pages.cpu().numpy(), page, heads, dim)
    for which, rows in ((0, turned[:, heads * group:]), (1, x[:, heads * (group + 1):])):
        code, d = R.quantize_q4(rows)
        at = table[seq[live], slot[live] // page], slice(None), slot[live] % page
        assert np.array_equal(got[which][at], code[live] - 8) and np.array_equal(got[2 + which][at], d[live])
        stands = ((code - 8) * np.repeat(d.astype(np.float32), 32, -1)).astype(np.float16)
        assert np.array_equal(kv[which].cpu().numpy(), np.where(live[:, None, None], stands, 0))


def test_append_at_bad_positions():
    cache, pages = make_cache(2, 16, 1, 64, [[0, 1]])
    x = torch.ones(4, 64, device="cuda")
    i32 = lambda v: dev(np.array(v, np.int32))  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kval = torch.zeros(4, 1, 64, dtype=torch.float16, device="cuda")
    rope = dev(R.rope_table(10, 64))
    Z.kv_append_q4_0(cache, x, x, i32([0] * 4), i32([3, 4, 5, 6]), rope=rope, rope_pos=i32([-1, 10, 9, 1 << 30]), k_val=kval, status=status)
    assert status.item() == 1 and kval.isnan().all(-1).flatten().tolist() == [True, True, False, True]
    # without a rotation its positions are not looked at
    status.zero_()
    Z.kv_append_q4_0(cache, x, x, i32([0] * 4), i32([3, 4, 5, 6]), rope_pos=i32([-1, 10, 9, 1 << 30]), k_val=kval, status=status)
    assert status.item() == 0 and not kval.isnan().any()


# ------------------------------------------------------------------ together
def test_a_run_of_them_together():
    """Prompts, then steps that draft trees, verify them, keep a path and count weights, then an eviction and one more step:
    the cache's contents, the attention and the weights against one line of tokens that is kept on the host."""
    rng = np.random.default_rng(12)
    heads, group, dim, page, n_seq, budget = 2, 4, 128, 16, 3, 64
    hq, cap = heads * group, 16
    rope_rows = 400
    rope = R.rope_table(rope_rows, dim)
    table = rng.permutation(n_seq * cap).reshape(n_seq, cap)
    cache, _ = make_cache(n_seq * cap, page, heads, dim, table, fill=0)
    per = 12
    cut_table = rng.permutation(n_seq * per).reshape(n_seq, per)
    cut, _ = make_cache(n_seq * per, page, heads, dim, cut_table, fill=0)
    lens = [100, 37, 150]            # tokens of the line that the cache holds
    truth = list(lens)               # positions that the sequences have had
    held_k, held_v = [[] for _ in range(n_seq)], [[] for _ in range(n_seq)]  # the line's fp64 values, [head][dim] each
    sums = torch.zeros(n_seq, heads, 256, device="cuda")
    want_sums = np.zeros((n_seq, heads, 256))
    rd = dev(rope)

    def append(c, counts, slots, turns):
        n = sum(counts)
        x = rng.standard_normal((n, hq + 2 * heads, dim)).astype(np.float32)
        q, k, v = (dev(t) for t in np.split(x, [hq, hq + heads], 1))
        kv = [torch.empty(n, heads, dim, dtype=torch.float16, device="cuda") for _ in range(2)]
        seq = np.repeat(np.arange(n_seq), counts).astype(np.int32)
        out = Z.kv_append_q4_0(c, k, v, dev(seq), dev(slots.astype(np.int32)), q=q, rope=rd, k_val=kv[0], v_val=kv[1],
                               rope_pos=dev(turns.astype(np.int32)))
        turned = R.rotate(x[:, :hq + heads], rope, turns, True)
        assert np.array_equal(out.cpu().numpy(), turned[:, :hq])
        vals = []
        for rows in (turned[:, hq:], x[:, hq + heads:]):
            code, d = R.quantize_q4(rows)
            vals.append((code - 8) * np.repeat(d.astype(np.float64), 32, -1))
        return out, turned[:, :hq], vals

    def verify(c, counts, masks):
        """Appends, attends, counts; returns the new tokens' values."""
        first = np.concatenate(([0], np.cumsum(counts)))
        depth = np.concatenate([m.sum(1) - 1 for m in masks])
        slots = np.concatenate([lens[s] + np.arange(counts[s]) for s in range(n_seq)])
        turns = np.repeat(truth, counts) + depth
        q, qh, vals = append(c, counts, slots, turns)
        now = [lens[s] + counts[s] for s in range(n_seq)]
        lse, words = torch.empty(len(depth), hq, device="cuda"), -(-max(counts) // 32)
        seen, starts, ld = dev(T.pack(masks, words)), dev(first.astype(np.int32)), dev(np.array(now, np.int32))
        out = Z.attn_tree_q4_0(c, q, starts, ld, max(counts), max(now), seen=seen, lse=lse).double().cpu().numpy()
        Z.attn_weights_q4_0(c, q, starts, ld, lse, max(counts), max(now), seen=seen, sums=sums, out=sums)
        got_lse = lse.double().cpu().numpy()
        for s in range(n_seq):
            kk, vv = ([np.stack([t[h] for t in line[s]] + [vals[w][first[s] + i][h] for i in range(counts[s])]) for h in range(heads)]
                      for w, line in ((0, held_k), (1, held_v)))
            want_sums[s, :, lens[s]:now[s]] = 0
            for i in range(counts[s]):
                row, see = first[s] + i, T.visible(now[s], counts[s], i, masks[s])
                for h in range(hq):
                    score = kk[h // group][see] @ qh[row, h].astype(np.float64) * dim ** -0.5
                    p = np.exp(score - score.max())
                    # the bounds of test_tree_gpu.py, with what the values here reach
                    reach = dim ** -0.5 * (np.abs(kk[h // group][see]).reshape(-1, 4, 32).max(-1) @ np.abs(qh[row, h]).reshape(4, 32).sum(-1)).max()
                    big = p / p.sum() @ np.abs(vv[h // group][see]).reshape(-1, 4, 32).max(-1)
                    err = np.abs(out[row, h] - p @ vv[h // group][see] / p.sum())
                    assert np.all(err <= np.repeat(big, 32) * (2 * 2.0 ** -19 * reach + 2.0 ** -17))
                    want_sums[s, h // group, :now[s]][see] += np.exp(score - got_lse[row, h])
        return vals, first

    def accept(c, counts, masks, vals, first):
        paths = []
        for s in range(n_seq):
            leaf = int(rng.integers(0, counts[s]))
            paths.append(np.flatnonzero(masks[s][leaf]))
        path = np.full((n_seq, max(map(len, paths))), 0, np.int32)
        for s, p in enumerate(paths):
            path[s, :len(p)] = p
        new = Z.kv_accept_q4_0(c, dev(np.array(lens, np.int32)), dev(path), dev(np.array([len(p) for p in paths], np.int32)), sums=sums)
        for s, p in enumerate(paths):
            for i in p:
                held_k[s].append(vals[0][first[s] + i])
                held_v[s].append(vals[1][first[s] + i])
            want_sums[s][:, lens[s]:lens[s] + len(p)] = want_sums[s][:, lens[s] + p]
            lens[s] += len(p)
            truth[s] += len(p)
        assert new.tolist() == lens

    # prompts: chains
    counts = list(lens)
    n0 = np.concatenate([np.arange(n) for n in counts])
    _, _, vals = append(cache, counts, n0, n0)
    at = 0
    for s in range(n_seq):
        held_k[s] += list(vals[0][at:at + counts[s]])
        held_v[s] += list(vals[1][at:at + counts[s]])
        at += counts[s]
    for step in range(3):
        counts = [5, 9, 12] if step < 2 else [1, 1, 33]
        masks = [T.tree_mask(n, rng) for n in counts]
        vals, first = verify(cache, counts, masks)
        accept(cache, counts, masks, vals, first)
    got = sums.double().cpu().numpy()
    for s in range(n_seq):
        # three steps of up to 132 rows a kv head: far below the bounds of a single one's terms
        assert np.abs(got[s, :, :lens[s]] - want_sums[s, :, :lens[s]]).max() < 2.0 ** -18 * 400 * want_sums[s].max()
    host = sums.cpu().numpy()
    out, new = torch.zeros_like(sums), torch.empty(n_seq, dtype=torch.int32, device="cuda")
    index = Z.kv_evict_q4_0(cache, cut, dev(np.array(lens, np.int32)), sums, budget, max(lens), sinks=2, recent=8, sums_out=out, len_out=new)
    want = T.evict_index(host, lens, budget, 2, 8)
    assert np.array_equal(index.cpu().numpy(), want)
    for s in range(n_seq):
        m = min(lens[s], budget)
        for line in (held_k, held_v):
            line[s] = [np.stack([line[s][want[s, h, j]][h] for h in range(heads)]) for j in range(m)]
        for h in range(heads):
            want_sums[s, h, :m] = want_sums[s, h][want[s, h, :m]]
        lens[s] = m
    assert new.tolist() == lens
    sums = out
    for _ in range(2):
        counts = [3, 1, 7]
        masks = [T.tree_mask(n, rng) for n in counts]
        vals, first = verify(cut, counts, masks)
        accept(cut, counts, masks, vals, first)
    assert Z.device_status() == 0


def test_they_run_as_a_graph():
    """A captured step (append, attention, weights, acceptance, eviction) replays on other inputs as the calls one by one."""
    rng = np.random.default_rng(4)
    heads, group, dim, page, n = 2, 2, 128, 16, 6
    lens = [60, 90]
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    to_table = np.arange(8).reshape(2, 4)
    masks = [T.tree_mask(n, rng) for _ in lens]
    i32 = lambda v: dev(np.array(v, np.int32))  # noqa: E731
    seen, starts, ld = dev(T.pack(masks, 1)), i32([0, n, 2 * n]), i32(lens)
    base, path, count = i32([v - n for v in lens]), i32([[0, 2, 5], [1, 3, 4]]), i32([3, 2])
    seq, slot = i32([0] * n + [1] * n), i32(list(range(lens[0] - n, lens[0])) + list(range(lens[1] - n, lens[1])))
    turn = i32(rng.integers(0, 300, 2 * n))
    rope = dev(R.rope_table(300, dim))
    x = torch.empty(2 * n, (2 + group) * heads * dim, device="cuda")
    q, k, v = x.split((heads * group * dim, heads * dim, heads * dim), 1)
    old = torch.rand(2, heads, 96, device="cuda")
    ws = Z.attn_q4_0_workspace(cache, heads * group, n, 90)

    def step(cache, to, r, stream=None):
        Z.kv_append_q4_0(cache, k, v, seq, slot, q=q, q_out=r["q"], rope=rope, rope_pos=turn, stream=stream)
        Z.attn_tree_q4_0(cache, r["q"], starts, ld, n, 90, seen=seen, lse=r["lse"], out=r["out"], workspace=ws, stream=stream)
        Z.attn_weights_q4_0(cache, r["q"], starts, ld, r["lse"], n, 90, seen=seen, sums=old, out=r["sums"], stream=stream)
        Z.kv_accept_q4_0(cache, base, path, count, sums=r["sums"], len_out=r["len"], stream=stream)
        Z.kv_evict_q4_0(cache, to, r["len"], r["sums"], 50, 90, sinks=1, recent=5, index=r["index"], sums_out=r["kept"], len_out=r["new"],
                        stream=stream)

    def results():
        e = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        return {"q": e(2 * n, heads * group, dim), "lse": e(2 * n, heads * group), "out": e(2 * n, heads * group, dim), "sums": e(2, heads, 96),
                "len": e(2, t=torch.int32), "index": e(2, heads, 50, t=torch.int32), "kept": e(2, heads, 50), "new": e(2, t=torch.int32)}
    to, _ = make_cache(8, page, heads, dim, to_table, fill=0)
    got, side = results(), torch.cuda.Stream()
    x.normal_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step(cache, to, got, side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(cache, to, got, side)
    for _ in range(3):
        torch.cuda.synchronize()
        x.normal_()
        old.uniform_()
        turn.copy_(i32(rng.integers(0, 300, 2 * n)))
        cache.pages.copy_(dev(pages))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        alone, want = Z.KVCache(dev(pages), page, heads, dim, dev(table)), results()
        to2, _ = make_cache(8, page, heads, dim, to_table, fill=0)
        step(alone, to2, want)
        torch.cuda.synchronize()
        assert torch.equal(alone.pages, cache.pages) and torch.equal(to2.pages, to.pages)
        for name in want:
            assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads, group, new", [(2, 4, 9), (1, 1, 65), (2, 8, 16), (1, 5, 129)])
def test_weights_many_columns(dim, heads, group, new):
    """36 to 645 columns: blocks of 64 that are full, nearly empty or one more than full; lengths around 128 tokens."""
    run_weights(np.random.default_rng(dim + new), [new, 127 + new, 128, 129, 700], [new, new, min(new, 128), 1, new - 1], 48, heads, group,
                dim, masks="tree" if new != 65 else None, window=0 if new < 100 else 150)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_weights_of_large_scales(dim):
    """Scales of 2^13 and more among 128 tokens (their operand in units of 16), small queries: the bound counts the keys' size."""
    rng = np.random.default_rng(dim)
    page, n, new, group = 32, 200, 12, 4
    cache, pages, table = random_cache(rng, [n], page, 1, dim)
    for at in (5, 130, 199):
        R.put(pages, page, 1, dim, table[0, at // page], at % page, 0, 0, rng.integers(0, 16, dim),
              np.linspace(8000, 60000, dim // 32).astype(np.float16))
    cache = Z.KVCache(dev(pages), page, 1, dim, dev(table))
    q = (2e-5 * rng.standard_normal((new, group, dim))).astype(np.float32)
    starts, ld, lse = dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32)), torch.empty(new, group, device="cuda")
    Z.attn_tree_q4_0(cache, dev(q), starts, ld, new, n, lse=lse)
    out = Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, new, n).double().cpu().numpy()
    k, _ = R.values(pages, page, 1, dim)
    want, tol = T.weights(q, [0, new], [n], table, k, page, dim ** -0.5, lse.double().cpu().numpy())
    # the other tokens' scales count to 2^-21 of themselves where they share an operand: 2^-21 P, within 2^-18 P
    assert np.all(np.abs(out - want) <= 2.0 ** -18 * tol + 1e-30)


def test_weights_of_a_prompts_chunk():
    """Two CTAs on some SMs, each with more blocks of columns than it has places for; the same bits again."""
    rng = np.random.default_rng(77)
    cache, q, starts, ld, lse, had, out = run_weights(rng, [3000], [256], 64, 8, 2, 128)
    for _ in range(3):
        again = torch.full_like(out, -7.0)
        Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, 256, 3000, sums=had, out=again)
        assert torch.equal(again, out)
    assert Z.device_status() == 0


@pytest.mark.parametrize("heads, group, dim, new, length", [(8, 4, 128, 15, 5200), (8, 2, 64, 31, 5200), (8, 4, 256, 12, 2600)])
def test_weights_of_a_middling_number_of_columns(heads, group, dim, new, length):
    """25 to 64 columns over more tokens than the tall kernel's CTAs take at once: sixteen groups of four at most."""
    run_weights(np.random.default_rng(dim), [length, 40], [new, new - 3], 64, heads, group, dim, masks="tree")


def test_pages_past_32_bits():
    """A cache of more than 2^32 bytes whose sequences lie in its last pages: what the same pages give at its start."""
    rng = np.random.default_rng(3)
    page, heads, dim, lens = 1024, 8, 256, [1500, 100]
    small, pages, table = random_cache(rng, lens, page, heads, dim, spare=0)
    per = Z.kv_page_bytes(page, heads, dim)
    n_pages, far = len(pages) // per, (1 << 32) // per + 3
    big = torch.empty((far + n_pages + 4) * per, dtype=torch.uint8, device="cuda")
    big[far * per:(far + n_pages) * per].copy_(small.pages)
    there = Z.KVCache(big, page, heads, dim, dev(np.where(table >= 0, table + far, -1).astype(np.int32)))
    i32 = lambda v: dev(np.array(v, np.int32))  # noqa: E731
    n = 5
    q, starts, ld = dev(rng.standard_normal((2 * n, 2 * heads, dim)).astype(np.float32)), i32([0, n, 2 * n]), i32(lens)
    seen, had = dev(T.pack([T.tree_mask(n, rng) for _ in lens], 1)), torch.rand(2, heads, 1500, device="cuda")
    base, path, count = i32([v - n for v in lens]), i32([[0, 2, 4], [1, 3, 0]]), i32([3, 2])
    results = []
    for cache, buffer, first in ((small, torch.zeros(2 * per, dtype=torch.uint8, device="cuda"), 0), (there, big, far + n_pages)):
        buffer[first * per:(first + 2) * per] = 0
        to = Z.KVCache(buffer, page, heads, dim, i32([[first + 1], [first]]))
        lse = torch.empty(2 * n, 2 * heads, device="cuda")
        out = Z.attn_tree_q4_0(cache, q, starts, ld, n, 1500, seen=seen, lse=lse)
        w = Z.attn_weights_q4_0(cache, q, starts, ld, lse, n, 1500, seen=seen, sums=had)
        new = Z.kv_accept_q4_0(cache, base, path, count, sums=w)
        index = Z.kv_evict_q4_0(cache, to, new, w, 700, 1500, sinks=2, recent=9)
        held = cache.pages if cache is small else big[far * per:(far + n_pages) * per]
        results.append((out, lse, w, new, index, held.clone(), buffer[first * per:(first + 2) * per].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert Z.device_status() == 0


def test_several_streams_at_once():
    """The same chain of calls on streams of their own, with buffers of their own, as alone."""
    rng = np.random.default_rng(6)
    jobs = []
    for dim, heads, group, n, length in ((128, 8, 4, 16, 3000), (256, 2, 8, 12, 1500), (64, 4, 1, 1, 4000)):
        cache, _, _ = random_cache(rng, [length, length // 2], 64, heads, dim)
        e = lambda *s, t=torch.float32: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        q = dev(rng.standard_normal((2 * n, heads * group, dim)).astype(np.float32))
        size = Z.attn_weights_q4_0_workspace_bytes(cache, heads * group, 2 * n, n)
        jobs.append(dict(cache=cache, n=n, length=length, q=q, starts=dev(np.array([0, n, 2 * n], np.int32)),
                         ld=dev(np.array([length, length // 2], np.int32)), seen=dev(T.pack([T.tree_mask(n, rng) for _ in range(2)], 1)),
                         had=torch.rand(2, heads, length, device="cuda"), lse=e(2 * n, heads * group), out=e(*q.shape), sums=e(2, heads, length),
                         index=e(2, heads, 300, t=torch.int32), kept=e(2, heads, 300), ws=Z.attn_q4_0_workspace(cache, heads * group, n, length),
                         ww=e(max(16, size), t=torch.uint8), to=make_cache(10, 64, heads, dim, np.arange(10).reshape(2, 5), fill=0)[0]))

    def chain(j, stream):
        for _ in range(8):
            Z.attn_tree_q4_0(j["cache"], j["q"], j["starts"], j["ld"], j["n"], j["length"], seen=j["seen"], lse=j["lse"], out=j["out"],
                             workspace=j["ws"], stream=stream)
            Z.attn_weights_q4_0(j["cache"], j["q"], j["starts"], j["ld"], j["lse"], j["n"], j["length"], seen=j["seen"], sums=j["had"],
                                out=j["sums"], workspace=j["ww"], stream=stream)
            Z.kv_evict_q4_0(j["cache"], j["to"], j["ld"], j["sums"], 300, j["length"], sinks=3, recent=50, index=j["index"],
                            sums_out=j["kept"], stream=stream)

    names = ("lse", "out", "sums", "index", "kept")
    alone = []
    for j in jobs:
        chain(j, torch.cuda.current_stream())
        torch.cuda.synchronize()
        alone.append([j[k].clone() for k in names] + [j["to"].pages.clone()])
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(4):
        for j in jobs:
            for k in names:
                j[k].zero_()
        torch.cuda.synchronize()
        for j, stream in zip(jobs, streams):
            chain(j, stream)
        torch.cuda.synchronize()
        for j, want in zip(jobs, alone):
            assert all(torch.equal(a, b) for a, b in zip([j[k] for k in names] + [j["to"].pages], want))
    assert Z.device_status() == 0
