"""Lengths at the end of 32 bits: a page table whose entries all name one page holds them."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests.test_block_ops_gpu import dev, random_cache

pytestmark = pytest.mark.gpu

MOST = 0x7FFFFF00


@pytest.mark.parametrize("group, bound", [(4, 2.0 ** -6), (16, 2.0 ** -6), (24, 2.0 ** -2)])
def test_the_longest_sequence_and_one_too_long(group, bound):
    """Every page being the same, a sequence of whole pages has the result of one page. The terms, 2^31, are added one after
    another by a lane, 2^17 of them (tcgen05: by a thread, 2^21.8), each time with an error below 2^-24 of the sum, for the sum
    of p and for that of p v."""
    rng = np.random.default_rng(group)
    page, heads, dim = 1024, 1, 64
    one, pages, _ = random_cache(rng, [page], page, heads, dim, spare=0)
    first = int(one.page_table[0, 0])
    table = torch.full((1, 1 << 21), first, dtype=torch.int32, device="cuda")
    cache = Z.KVCache(one.pages, page, heads, dim, table)
    q = rng.standard_normal((1, group, dim)).astype(np.float32)
    q_start = dev(np.array([0, 1], np.int32))
    k, v = R.values(pages, page, heads, dim)
    want, _, tol = R.attention(q, [0, 1], [page], np.array([[first]]), k, v, page, dim ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for n in (MOST // page * page, 2 ** 31 - 1, MOST + 1):
        out = Z.attn_q4_0(cache, dev(q), q_start, dev(np.array([n], np.int32)), 1, 2 ** 31 - 1, status=status)
        if n <= MOST:
            assert status.item() == 0
            assert (np.abs(out.double().cpu().numpy() - want) <= tol * bound).all()
        else:  # past what the tokens' numbers hold: refused as any bad sequence
            assert status.item() == 1 and out.isnan().all()
        status.zero_()
