"""Sizes at the end of 32 bits, without a GPU: the kernels' counters go a step past them."""
import ctypes

import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests.test_block_ops_cpu import FAKE, L, _cache  # noqa: F401
from tests.test_gave_up_waits_cpu import source
from tests.test_tree_cpu import _evict


def _call(L, budget):  # noqa: F811
    """One kv head of one sequence to a cache whose page table has room for 2^31 tokens and more."""
    one = dict(n_seq=1, n_kv_heads=1, head_dim=64)
    to = _cache(**one, pages=9 * FAKE, page_table=10 * FAKE, max_pages=1 << 22, page_tokens=1024)
    args = _evict(kv_len=2 * FAKE, sums=3 * FAKE, index=4 * FAKE, sums_out=None, len_out=None, status_dev=None, budget=budget)
    return L.zdmmv_kv_evict_q4_0(ctypes.byref(_cache(**one)), ctypes.byref(to), ctypes.byref(args), None)


def test_evict_refuses_budgets_at_the_end_of_32_bits(L):  # noqa: F811
    """The places of index are counted in steps of a cluster's threads: from a budget of 2^31 - 8192 on the last step had no number, and
    the next place was before the array."""
    for budget in (0x7fff0001, 0x7fffe000, 0x7fffffff):
        assert _call(L, budget) == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would run")
def test_evict_takes_the_largest_budget(L):  # noqa: F811
    assert _call(L, 0x7fff0000) not in (1, 2, 3)


def test_the_largest_step():
    """What is left above the bound is more than a cluster's threads."""
    import re
    text = source("zdmmv_kv_keep.cu")
    value = lambda name: int(re.search(rf"\b{name} = (0x[0-9a-f]+|\d+)", text).group(1), 0)  # noqa: E731
    assert value("kPickMost") + value("kPickThreads") * value("kPickCluster") < 1 << 31


def test_the_binding_makes_a_workspace_where_one_is_needed(L):  # noqa: F811
    for kv, group, dim, n_tok, most in [(k, g, d, t, m) for k in (1, 2, 8) for g in (1, 3, 4, 8, 24, 25, 64) for d in (64, 128, 256)
                                        for t in (0, 1, 5, 6, 24, 25, 100) for m in (1, 3, 6, 7, 24, 25, 200)]:
        cache = _cache(n_kv_heads=kv, head_dim=dim)
        need = L.zdmmv_attn_weights_q4_0_workspace_bytes(ctypes.byref(cache), kv * group, n_tok, most)
        assert (need > 0) == (kv * group * min(n_tok, most) > Z._FEW_COLUMNS * kv), (kv, group, dim, n_tok, most)
