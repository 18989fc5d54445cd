"""Eviction that writes the new lengths over the old ones (len_out is kv_len): what it gives with lengths of their own, on one CTA a kv
head and on clusters. Everything here is whole numbers and bytes that move: equal."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests.test_block_ops_gpu import dev, make_cache, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens, budget, most, bad", [([700, 90, 64, 0, 3, 650], 64, 700, 4), ([30000, 21000, 500, 400], 400, 30000, 2),
                                                     ([70001, 33333], 16000, 70001, 1)])
def test_evict_in_place(lens, budget, most, bad):
    rng = np.random.default_rng(budget)
    heads, dim, page = 8, 64, 64
    cache, _, _ = random_cache(rng, lens, page, heads, dim)
    sums = torch.rand(len(lens), heads, most, device="cuda")
    per = -(-budget // page)
    table = rng.permutation(len(lens) * per).reshape(len(lens), per)

    def evict(now, len_out):
        to, _ = make_cache(len(lens) * per, page, heads, dim, table, seed=5)
        status, kept = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((len(lens), heads, budget), -7.0, device="cuda")
        index = Z.kv_evict_q4_0(cache, to, now, sums, budget, most, sinks=1, recent=9, sums_out=kept, len_out=len_out, status=status)
        return index, kept, to.pages, len_out, status

    for wrong in (None, -1, most + 1):
        given = list(lens)
        if wrong is not None:
            given[bad] = wrong
        want = evict(dev(np.array(given, np.int32)), torch.full((len(lens),), -9, dtype=torch.int32, device="cuda"))
        assert want[3].tolist() == [-1 if n == wrong else min(n, budget) for n in given] and want[4].item() == (wrong is not None)
        for _ in range(20):
            now = dev(np.array(given, np.int32))
            assert all(torch.equal(a, b) for a, b in zip(evict(now, now), want))
    # cut back again: nothing more goes, and the lengths stay
    again = want[3].clone()
    again[bad] = 0
    keep = again.clone()
    assert torch.equal(evict(again, again)[3], keep)
    assert Z.device_status() == 0
