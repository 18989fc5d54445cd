"""A key with an infinite scale (a value past 524000 is stored so) whose scores are -infinity has no weight, however many columns the
call has beside a multiple of four; the others have what they have without it."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import tree_ref as T
from tests.test_attention_huge_scores_gpu import put_k
from tests.test_block_ops_gpu import dev, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("group, new", [(1, 1), (2, 1), (3, 1), (4, 1), (5, 1), (2, 3), (7, 1), (5, 3)])
def test_a_score_of_minus_infinity(dim, group, new):
    rng = np.random.default_rng(dim + group)
    heads, page, n, at = 2, 32, 100, 37
    cache, pages, table = random_cache(rng, [n], page, heads, dim)
    u = np.where(rng.random(dim) < 0.5, 1, -1)
    q = rng.standard_normal((new, heads * group, dim)).astype(np.float32)
    q[..., :32] = -u[:32] * np.abs(q[..., :32])
    scale = np.full(dim // 32, 0.1, np.float16)
    scale[0] = np.inf
    for h in range(heads):
        put_k(pages.reshape(-1, heads, page // 16, 18 * dim)[table[0, at // page], h, at % page // 16], dim, at % 16, (8 + 7 * u).astype(np.uint8), scale)
    cache.pages.copy_(dev(pages))
    starts, ld, lse = dev(np.array([0, new], np.int32)), dev(np.array([n], np.int32)), torch.empty(new, heads * group, device="cuda")
    seen = np.ones((new, new), bool)
    seen[0] = seen[0] & (np.arange(new) == 0)
    bits = dev(T.pack([seen], 1))
    Z.attn_tree_q4_0(cache, dev(q), starts, ld, new, n, seen=bits, lse=lse)
    assert torch.isfinite(lse).all()
    out = Z.attn_weights_q4_0(cache, dev(q), starts, ld, lse, new, n, seen=bits)
    assert not out[0, :, at].any()
    assert torch.isfinite(out).all() and (out.double().sum(-1) - new * group).abs().max() < new * group * 2.0 ** -18 * 128
    assert Z.device_status() == 0
