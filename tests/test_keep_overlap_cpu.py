"""Lengths that eviction and the accepted path write over those that they read: what is allowed and what is refused, without a GPU."""
import ctypes

import pytest
import torch

from tests.test_block_ops_cpu import FAKE, L, _cache  # noqa: F401
from tests.test_gave_up_waits_cpu import block, source
from tests.test_tree_cpu import _accept, _evict


def _evict_call(L, **k):  # noqa: F811
    to = _cache(pages=9 * FAKE, page_table=10 * FAKE)
    args = _evict(**{**dict(kv_len=2 * FAKE, sums=3 * FAKE, index=4 * FAKE, sums_out=5 * FAKE, len_out=6 * FAKE, status_dev=7 * FAKE), **k})
    return L.zdmmv_kv_evict_q4_0(ctypes.byref(_cache()), ctypes.byref(to), ctypes.byref(args), None)


def test_evict_refuses_lengths_that_overlap_in_part(L):  # noqa: F811
    """Two sequences: a shift by one of them overlaps."""
    for shift in (-4, 4):
        assert _evict_call(L, len_out=2 * FAKE + shift) == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would run")
def test_evict_takes_lengths_in_place(L):  # noqa: F811
    for len_out in (None, 6 * FAKE, 2 * FAKE, 2 * FAKE + 8, 2 * FAKE - 8):
        assert _evict_call(L, len_out=len_out) not in (1, 2, 3)


def test_evict_writes_a_length_where_one_thread_alone_reads_it():
    """The choice's CTAs all read a sequence's length, in no order among them: what they write is none. The move, which runs after all of
    them, has one thread a sequence that reads it and writes it."""
    text = source("zdmmv_kv_keep.cu")
    pick = block(text, text.index("kv_pick_kernel(KeepArgs a)"))
    move = block(text, text.index("kv_gather_kernel(KeepArgs a, int64_t n_jobs)"))
    assert "a.kv_len[seq]" in pick and "len_out" not in pick
    own = block(move, move.index("if (a.len_out && tile == 0 && kvh == 0 && lane == 0)"))
    assert move.count("kv_len") == own.count("a.kv_len[seq]") == 1 and move.count("a.len_out[seq]") == own.count("a.len_out[seq]") == 1
    assert move.index("block_op_wait()") < move.index("a.kv_len[seq]") < move.index("a.len_out[seq]")


def _accept_call(L, **k):  # noqa: F811
    args = _accept(**{**dict(base=2 * FAKE, path=3 * FAKE, n_path=4 * FAKE, len_out=5 * FAKE, status_dev=6 * FAKE, sums=7 * FAKE), **k})
    return L.zdmmv_kv_accept_q4_0(ctypes.byref(_cache()), ctypes.byref(args), None)


@pytest.mark.parametrize("what, size", [(2 * FAKE, 8), (4 * FAKE, 8), (3 * FAKE, 2 * 8 * 4)])
def test_accept_refuses_lengths_over_its_inputs(L, what, size):  # noqa: F811
    """base, n_path (two sequences) and path (of eight places each), from the first byte to the last."""
    for at in (what - 4, what, what + size - 4):
        assert _accept_call(L, len_out=at) == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would run")
def test_accept_takes_lengths_beside_its_inputs(L):  # noqa: F811
    for at in (None, 5 * FAKE, 2 * FAKE - 8, 2 * FAKE + 8, 3 * FAKE - 8, 3 * FAKE + 64, 4 * FAKE + 8):
        assert _accept_call(L, len_out=at) not in (1, 2, 3)
