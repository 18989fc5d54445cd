"""What a row does not see has no part in it, whatever it is: infinities and NaN in the cache (a value past fp16's range times 8 is
stored as one) before the window and among the tokens after the row's own."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests import test_attention_columns_gpu as C
from tests.test_attention_scales_gpu import FORMS, TALL, attend
from tests.test_block_ops_gpu import check_attention, dev, make_cache, random_cache

pytestmark = pytest.mark.gpu


def spoil(pages, table, page, heads, dim, seq, tok, which, value, blocks):
    """Scales of a token's K (0) or V (1), in these blocks, become `value`."""
    t = pages.reshape(-1, heads, page // 16, 18 * dim)
    at = R.tile_index(dim)[2][tok % 16][blocks]
    base = (16 + which) * dim
    row = t[table[seq, tok // page], :, tok % page // 16, base:base + dim].copy().view(np.float16)
    row[:, at] = value
    t[table[seq, tok // page], :, tok % page // 16, base:base + dim] = row.view(np.uint8)


@pytest.mark.parametrize("dim, group, new", FORMS + TALL)
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_non_finite_tokens_that_rows_do_not_see(dim, group, new, value):
    rng = np.random.default_rng(dim + group + new)
    lens, heads, page, window = [40, 300], 2, 32, 25
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    spoilt = pages.copy()
    nb = dim // 32
    # every sequence: the last token that no row's window reaches, in all blocks, K and V; the new token before the last (if
    # there are two), V alone, in the last block
    for s, n in enumerate(lens):
        for which in (0, 1):
            spoil(spoilt, table, page, heads, dim, s, n - new - window, which, value, np.arange(nb))
        if new > 1:
            spoil(spoilt, table, page, heads, dim, s, n - 2, 1, value, np.array([nb - 1]))
    cache.pages.copy_(dev(spoilt))
    q = rng.standard_normal((2 * new, heads * group, dim)).astype(np.float32)
    out, q_start = attend(cache, q, lens, [new, new], window=window)
    k, v = R.values(pages, page, heads, dim)
    got = out.cpu().numpy().reshape(2, new, heads * group, dim)
    if new > 1:  # the rows that see the spoilt new token have lost its block, and nothing else
        assert not np.isfinite(got[:, -2:, :, -32:]).any()
        want = R.attention(q, q_start, lens, table, k, v, page, dim ** -0.5, window)[0].reshape(got.shape)
        got[:, -2:, :, -32:] = want[:, -2:, :, -32:]
    out.copy_(dev(got.reshape(out.shape)))
    args = (out, q, q_start, lens, table, pages, page, heads, dim)
    if (dim, group, new) in TALL:
        C.check(*args, dim ** -0.5, window)
    else:
        check_attention(*args, window=window)


def test_a_value_that_the_append_stores_as_infinity():
    page, heads, dim, n = 32, 2, 128, 20
    g = torch.Generator("cuda").manual_seed(3)
    table = np.arange(2)[None]
    k, v = (torch.randn(n, heads, dim, device="cuda", generator=g) for _ in range(2))
    v[n - 1, :, 5] = 6e5
    seq, pos = torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda")
    q = torch.randn(4, heads * 8, dim, device="cuda", generator=g)
    outs = []
    for last in (n, n - 1):  # with that token, and without it
        cache, _ = make_cache(2, page, heads, dim, table)
        Z.kv_append_q4_0(cache, k[:last].contiguous(), v[:last].contiguous(), seq[:last], pos[:last])
        new = 4 - (n - last)
        outs.append(Z.attn_q4_0(cache, q[:new].contiguous(), dev(np.array([0, new], np.int32)), dev(np.array([last], np.int32)), new, n))
    assert torch.isfinite(outs[1]).all() and not torch.isfinite(outs[0][3, :, :32]).any()
    assert torch.allclose(outs[0][:3], outs[1], rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dim, group, new", [(128, 4, 1), (64, 4, 3), (128, 8, 2), (192, 8, 5), (256, 16, 5), (64, 8, 8), (96, 8, 5),
                                             (128, 8, 16)])
@pytest.mark.parametrize("window", [0, 2000])
def test_non_finite_tokens_in_long_sequences(dim, group, new, window):
    """The same where a row's sums are joined from parts, some of which have such a token."""
    rng = np.random.default_rng(dim + group + new)
    lens, heads, page = [5003], 1, 64
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    spoilt, n, nb = pages.copy(), lens[0], dim // 32
    if window:
        spoil(spoilt, table, page, heads, dim, 0, n - new - window, 1, np.nan, np.arange(nb))
    if new > 1:
        spoil(spoilt, table, page, heads, dim, 0, n - 1, 1, np.inf, np.array([0]))
    cache.pages.copy_(dev(spoilt))
    q = rng.standard_normal((new, heads * group, dim)).astype(np.float32)
    out, q_start = attend(cache, q, lens, [new], window=window)
    if new > 1:
        assert not torch.isfinite(out[-1, :, :32]).any() and torch.isfinite(out[-1, :, 32:]).all()
        k, v = R.values(pages, page, heads, dim)
        want = R.attention(q, q_start, lens, table, k, v, page, dim ** -0.5, window)[0]
        out[-1, :, :32] = dev(want[-1, :, :32].astype(np.float32))
    args = (out, q, q_start, lens, table, pages, page, heads, dim)
    if dim <= 128 and group * new > 16:
        C.check(*args, dim ** -0.5, window)
    else:
        check_attention(*args, window=window)
