"""Scores far past 2^24, where a float's step is more than a softmax can show, up to the end of fp32's range: one token has all the
weight, and the result is its V (to the bounds' 2^-17)."""
import functools

import numpy as np
import pytest

from tests import block_ref as R
from tests.test_attention_scales_gpu import FORMS, TALL, attend
from tests.test_block_ops_gpu import dev, random_cache

pytestmark = pytest.mark.gpu


tile_index = functools.cache(R.tile_index)


def put_k(tile, dim, tok, codes, scale):
    """R.put of one token's K in one tile (bytes), without a loop."""
    index = tile_index(dim)
    n = index[0][tok]
    for high in (0, 1):
        at = n[n % 2 == high] // 2
        tile[at] = (tile[at] & (0x0F if high else 0xF0)) | (codes[n % 2 == high] << 4 * high)
    tile[16 * dim:17 * dim].view(np.float16)[index[2][tok]] = scale


@pytest.mark.parametrize("dim, group, new", FORMS + TALL)
@pytest.mark.parametrize("size", [1e5, 1e7, 1e10, 1e22, 1e33, 1e35, -1e5, -1e7, -1e10, -1e22, -1e33, -1e35])
def test_the_largest_score_takes_all(dim, group, new, size):
    """Every token's K is the same direction u, of a length of its own, and q is size times u: scores of one sign, whose
    neighbours are 1 / 100 of their size apart or more."""
    takes_all(dim, group, new, size, [90, 37], 2, lambda n: np.linspace(0.05, 0.3, n))


@pytest.mark.parametrize("dim, group, new", [(128, 4, 1), (64, 8, 1), (192, 20, 5), (64, 8, 8), (128, 8, 16)])
@pytest.mark.parametrize("size", [1e7, 1e22, -1e22])
def test_the_largest_score_of_many_parts(dim, group, new, size):
    """The same over a length whose parts are joined; all but a few tokens are as long as one another."""
    def lengths(n):
        d = np.full(n, 0.2)
        d[:4] = 0.31, 0.3, 0.05, 0.06
        return d
    takes_all(dim, group, new, size, [4000], 1, lengths)


def takes_all(dim, group, new, size, lens, heads, lengths):
    rng = np.random.default_rng(dim + group)
    page = 32
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    u = np.where(rng.random((heads, dim)) < 0.5, 1, -1)
    d = np.zeros((len(lens), max(lens)))
    for s, n in enumerate(lens):
        d[s, :n] = rng.permutation(lengths(n))
        for tok in range(n):
            for h in range(heads):
                put_k(pages.reshape(-1, heads, page // 16, 18 * dim)[table[s, tok // page], h, tok % page // 16], dim, tok % 16,
                      (8 + 7 * u[h]).astype(np.uint8), np.float16(d[s, tok]))
    cache.pages.copy_(dev(pages))
    sign = 1 if size > 0 else -1
    q = np.repeat(size * u[None], group, 1).astype(np.float32) * np.ones((2 * new, 1, 1), np.float32)
    out, q_start = attend(cache, q, lens, [new, new])
    got = out.double().cpu().numpy().reshape(2, new, heads, group, dim)
    v = R.values(pages, page, heads, dim)[1]
    for s, n in enumerate(lens):
        for i in range(new):
            sees = n - (new - 1 - i)
            best = int(np.argmax(sign * d[s, :sees].astype(np.float16)))
            want = v[table[s, best // page], :, best % page]                    # [head][dim]
            tol = 2.0 ** -17 * np.repeat(np.abs(want).reshape(heads, -1, 32).max(-1), 32, -1)
            assert (np.abs(got[s, i] - want[:, None]) <= tol[:, None]).all()
