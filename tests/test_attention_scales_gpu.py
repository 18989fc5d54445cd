"""Attention over blocks whose scales differ by up to fp16's whole range, in every form of the kernel. The bounds are those of
tests/test_block_ops_gpu.py and (tcgen05) tests/test_attention_columns_gpu.py, which are each block's own: large values in one
block of 32 dimensions do not excuse errors in another."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests import test_attention_columns_gpu as C
from tests.test_block_ops_gpu import check_attention, dev, random_cache

pytestmark = pytest.mark.gpu

# (dimensions, group, new tokens): narrow, wide with one and two groups of columns, shared ring, fragments made once
FORMS = [(64, 4, 1), (128, 4, 1), (256, 2, 1), (96, 1, 3), (192, 4, 1), (64, 8, 1), (128, 8, 1), (96, 8, 1), (256, 7, 1),
         (192, 5, 1), (128, 16, 1), (64, 5, 3), (96, 12, 1), (192, 16, 1), (256, 16, 1), (192, 24, 1), (256, 8, 6),
         (192, 20, 5), (256, 10, 9)]
# ... and on tcgen05
TALL = [(64, 17, 1), (96, 8, 5), (128, 8, 16), (128, 40, 4)]


def setup(rng, lens, heads, dim, k_scales, v_scales, page=32):
    """A cache whose scales of K and V are given: functions of (tokens, heads, blocks) -> fp16 values."""
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    t = pages.reshape(-1, heads, page // 16, 18 * dim)
    at = R.tile_index(dim)[2]
    for s, n in enumerate(lens):
        for base, f in ((16 * dim, k_scales), (17 * dim, v_scales)):
            if f is None:
                continue
            sc = np.asarray(f(n, heads, dim // 32)).astype(np.float16)
            for tok in range(n):
                row = t[table[s, tok // page], :, tok % page // 16, base:base + dim].view(np.float16)
                row[:, at[tok % 16]] = sc[tok]
                t[table[s, tok // page], :, tok % page // 16, base:base + dim] = row.view(np.uint8)
    cache.pages.copy_(dev(pages))
    return cache, pages, table


def attend(cache, q, lens, new, **kw):
    q_start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Z.attn_q4_0(cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), max(new), max(lens), status=status, **kw)
    assert status.item() == 0
    return out, q_start


def check(dim, group, new, *args):
    if (dim, group, new) in TALL:
        C.check(*args, dim ** -0.5, 0)
    else:
        check_attention(*args)


@pytest.mark.parametrize("dim, group, new", FORMS + TALL)
@pytest.mark.parametrize("large", [2.0 ** 3, 2.0 ** 12, 2.0 ** 14.9])
def test_large_and_small_blocks_of_v(dim, group, new, large):
    """Every other block's scales are `large`, the others' 2^-12."""
    rng = np.random.default_rng(dim + group)
    lens, heads = [23, 300], 2

    def scales(n, h, nb):
        size = np.where((np.arange(nb) + np.arange(h)[:, None]) % 2, 2.0 ** -12, large)
        return size * rng.uniform(0.6, 1.0, (n, h, nb)) * rng.choice([-1, 1], (n, h, nb))
    cache, pages, table = setup(rng, lens, heads, dim, None, scales)
    q = (0.1 * rng.standard_normal((2 * new, heads * group, dim))).astype(np.float32)
    out, q_start = attend(cache, q, lens, [new, new])
    check(dim, group, new, out, q, q_start, lens, table, pages, 32, heads, dim)


@pytest.mark.parametrize("dim, group, new", FORMS + TALL)
def test_large_and_small_tokens_of_v(dim, group, new):
    """Some tokens' scales are 2^14, the others' 2^-2 (a block's scales 2^16 apart)."""
    rng = np.random.default_rng(dim + group)
    lens, heads = [40, 517], 2

    def scales(n, h, nb):
        size = np.where(rng.random((n, h, 1)) < 0.1, 2.0 ** 14, 2.0 ** -2)
        return size * rng.uniform(0.6, 1.0, (n, h, nb)) * rng.choice([-1, 1], (n, h, nb))
    cache, pages, table = setup(rng, lens, heads, dim, None, scales)
    q = (0.1 * rng.standard_normal((2 * new, heads * group, dim))).astype(np.float32)
    out, q_start = attend(cache, q, lens, [new, new])
    check(dim, group, new, out, q, q_start, lens, table, pages, 32, heads, dim)


@pytest.mark.parametrize("dim, group, new", FORMS)
def test_a_large_token_of_little_weight(dim, group, new):
    """A token's values are 2^27 times the others' and its weight e^-12: it is most of the sum all the same, and its weight has
    to be as exact as any."""
    rng = np.random.default_rng(dim * group)
    n, heads, page = 64, 1, 32
    cache, pages, table = random_cache(rng, [n], page, heads, dim)
    t = pages.reshape(-1, heads, page // 16, 18 * dim)
    big = 20
    c = 0.5
    score = -12.0 / (dim ** -0.5 * c * 7 * dim)               # of the scale of K: codes 15 stand for 7
    for tok in range(n):
        for which in range(2):
            codes = np.full(dim, 15) if which == 0 else rng.integers(0, 16, dim)
            size = (score if tok == big else 0.0) if which == 0 else (2.0 ** 15 if tok == big else 2.0 ** -12)
            sc = np.full(dim // 32, size) * (rng.uniform(0.6, 1.0, dim // 32) if which else 1.0)
            R.put(pages, page, heads, dim, table[0, tok // page], tok % page, 0, which, codes, sc.astype(np.float16))
    cache.pages.copy_(dev(pages))
    q = np.full((new, group, dim), c, np.float32)
    out, q_start = attend(cache, q, [n], [new])
    check_attention(out, q, q_start, [n], table, pages, page, heads, dim)
