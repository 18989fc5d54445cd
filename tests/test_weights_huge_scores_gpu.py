"""Weights of rows whose scores are so large that a float's step is more than a softmax can show, up to the end of fp32's range.

Bounds, in powers of two (S the score's size there, y that of lse): lse and its product carry four roundings, 2^-21.9 y; a score is off by
2^-19 S at most (tests/test_block_ops_gpu.py), here and in the kernel that made lse, and all of a token's products have one sign here, so that
S is y: 2^-17.9 y in all. The exponent is raised by 2^-17 (y - 2^20), which is more from y = 2^21 on: the token with all of a row's weight
has the exponent 0, and its weight is 1. Below, it lacks 2^-17.9 2^20 < 4.4 at most. The others' scores are 1 / 150 of S or
more below it, more than 2^12 with these sizes: their weights are 0."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests import tree_ref as T
from tests.test_attention_huge_scores_gpu import put_k
from tests.test_block_ops_gpu import dev, random_cache

pytestmark = pytest.mark.gpu

# one column to 24 (mma.sync), 25 to 256 (tcgen05)
FORMS = [(64, 1, 1), (128, 4, 1), (96, 3, 5), (256, 8, 3), (192, 5, 5), (64, 8, 8), (128, 8, 16), (256, 4, 20), (128, 16, 16)]


def weights_of(dim, group, new, size, lens, heads, lengths):
    """(out, how many rows each token has all the weight of), both [seq][head][token]."""
    rng = np.random.default_rng(dim + group)
    page = 32
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    u = np.where(rng.random((heads, dim)) < 0.5, 1, -1)
    count = np.zeros((len(lens), heads, max(lens)))
    for s, n in enumerate(lens):
        d = rng.permutation(lengths(n)).astype(np.float16)
        for tok in range(n):
            for h in range(heads):
                put_k(pages.reshape(-1, heads, page // 16, 18 * dim)[table[s, tok // page], h, tok % page // 16], dim, tok % 16,
                      (8 + 7 * u[h]).astype(np.uint8), d[tok])
        for i in range(new):
            count[s, :, np.argmax(np.sign(size) * d[:n - (new - 1 - i)].astype(np.float64))] += group
    cache.pages.copy_(dev(pages))
    q = dev(np.repeat(size * u[None], group, 1).astype(np.float32) * np.ones((len(lens) * new, 1, 1), np.float32))
    starts, ld = dev((new * np.arange(len(lens) + 1)).astype(np.int32)), dev(np.array(lens, np.int32))
    lse = torch.empty(q.shape[:2], device="cuda")
    Z.attn_tree_q4_0(cache, q, starts, ld, new, max(lens), lse=lse)
    out = Z.attn_weights_q4_0(cache, q, starts, ld, lse, new, max(lens))
    assert Z.device_status() == 0
    return out.double().cpu().numpy(), count


@pytest.mark.parametrize("dim, group, new", FORMS)
@pytest.mark.parametrize("size", [3e6, 1e7, 3e7, 1e10, 1e22, 1e35, -3e6, -1e7, -3e7, -1e10, -1e22, -1e35])
def test_the_largest_score_has_the_weight(dim, group, new, size):
    out, count = weights_of(dim, group, new, size, [90, 37], 2, lambda n: np.linspace(0.05, 0.3, n))
    assert np.array_equal(out, count)


@pytest.mark.parametrize("dim, group, new", FORMS)
@pytest.mark.parametrize("size", [1e5, 3e5, -1e6])
def test_scores_where_the_exponent_begins_to_be_raised(dim, group, new, size):
    out, count = weights_of(dim, group, new, size, [90, 37], 2, lambda n: np.linspace(0.05, 0.3, n))
    assert np.all(out <= count) and np.all(out >= 2.0 ** -4.4 * count)


@pytest.mark.parametrize("dim, group, new", FORMS)
@pytest.mark.parametrize("size", [1e7, 1e22, -1e22])
def test_the_largest_score_of_a_long_sequence(dim, group, new, size):
    """The attention's sums, and with them lse, are joined from parts."""
    def lengths(n):
        d = np.full(n, 0.2)
        d[:4] = 0.31, 0.3, 0.05, 0.06
        return d
    out, count = weights_of(dim, group, new, size, [3000], 1, lengths)
    assert np.array_equal(out, count)


@pytest.mark.parametrize("dim, group, new", FORMS)
def test_a_weight_is_one_at_most(dim, group, new):
    """One token that every row sees: its score is all of lse but for roundings; one that is no number stays so."""
    rng = np.random.default_rng(dim)
    heads, page, n = 2, 32, new
    cache, pages, table = random_cache(rng, [n], page, heads, dim)
    starts, ld = dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32))
    seen = torch.ones(new, 1, dtype=torch.int32, device="cuda")        # token 0 alone
    for size in (1.0, 100.0, 1e4):
        q = dev((size * rng.standard_normal((new, heads * group, dim))).astype(np.float32))
        lse = torch.empty(new, heads * group, device="cuda")
        Z.attn_tree_q4_0(cache, q, starts, ld, new, n, seen=seen, lse=lse)
        out = Z.attn_weights_q4_0(cache, q, starts, ld, lse, new, n, seen=seen)
        assert torch.all(out[0, :, 0] <= new * group) and torch.all(out[0, :, 0] > 0) and not out[0, :, 1:].any()
    tile = pages.reshape(-1, heads, page // 16, 18 * dim)[table[0, 0], 0, 0]
    put_k(tile, dim, 0, np.full(dim, 9), np.float16(np.nan))
    cache.pages.copy_(dev(pages))
    out = Z.attn_weights_q4_0(cache, q, starts, ld, torch.zeros_like(lse), new, n, seen=seen)
    assert torch.isnan(out[0, 0, 0]) and torch.isfinite(out[0, 1]).all() and not out[0, 0, 1:].any()


@pytest.mark.parametrize("dim, group, new", FORMS)
@pytest.mark.parametrize("size", [3e6, 3e7, 1e10, 1e30])
def test_queries_along_a_key(dim, group, new, size):
    """Random keys, each row's q along one that it sees: its products are positive, P within twice their sum. Where the raise is more than
    both scores' 2^-19 P and lse's roundings, and the largest score is alone by more than all of these, its weight is the row's."""
    rng = np.random.default_rng(dim + group)
    heads, page, n = 2, 32, 150
    cache, pages, table = random_cache(rng, [n], page, heads, dim)
    masks = [T.tree_mask(new, rng)]
    k, _ = R.values(pages, page, heads, dim)
    keys = k[table[0][np.arange(n) // page], :, np.arange(n) % page]      # [token][head][dim]
    q = np.zeros((new, heads, group, dim))
    for i in range(new):
        see = np.flatnonzero(T.visible(n, new, i, masks[0]))
        for h in range(heads):
            q[i, h] = size * keys[rng.choice(see, group), h]
    q = q.reshape(new, heads * group, dim).astype(np.float32)
    starts, ld, seen = dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32)), dev(T.pack(masks, 1))
    lse = torch.empty(new, heads * group, device="cuda")
    Z.attn_tree_q4_0(cache, dev(q), starts, ld, new, n, seen=seen, lse=lse)
    out = Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, new, n, seen=seen)[0].double().cpu().numpy()
    assert Z.device_status() == 0
    least, clear_rows = np.zeros((heads, n)), 0
    for i in range(new):
        see = T.visible(n, new, i, masks[0])
        for c in range(heads * group):
            h = c // group
            score = np.where(see, keys[:, h] @ q[i, c].astype(np.float64), -np.inf) * dim ** -0.5 / np.log(2)
            reach = (np.abs(keys[see, h]).reshape(-1, dim // 32, 32).max(-1) @ np.abs(q[i, c].astype(np.float64)).reshape(-1, 32).sum(-1)).max()
            err = 2.0 ** -18 * reach * dim ** -0.5 / np.log(2) + 2.0 ** -21.9 * np.abs(score[see]).max()
            best, raised = score.argmax(), 2.0 ** -17 * (score.max() - 2.0 ** 20)
            others = np.delete(score, best).max()
            if raised >= err and score.max() - others > err + raised + 160:   # 2^-160 is 0
                least[h, best] += 1
                clear_rows += 1
    assert clear_rows > 0.1 * new * heads * group  # of the inputs alone: 4 of 30 to 2 of 2
    assert np.all(out >= least) and np.all(out.sum(-1) >= least.sum(-1)) and np.all(out <= new * group)
