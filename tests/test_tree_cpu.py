"""The operators on drafted trees and eviction without a GPU: argument checks and structs."""
import ctypes

import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import test_block_ops_cpu as B
from tests.test_block_ops_cpu import FAKE, L, _attn, _cache, _header_fields  # noqa: F401


class _AttnTree(ctypes.Structure):
    _fields_ = [("seen", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("seen_words", ctypes.c_int32)]


@pytest.mark.parametrize("name, c, packed", [("zdmmv_attn_tree", _AttnTree, Z._ATTN_TREE)])
def test_packed_structs_match_the_header(name, c, packed):
    B.test_packed_structs_match_the_header(name, c, packed)


def _tree(**k):
    return _AttnTree(**{**dict(seen=FAKE, lse=FAKE, seen_words=1), **k})


@pytest.mark.parametrize("code, change", [
    (2, dict(seen_words=0)), (2, dict(seen_words=-1)), (2, dict(seen_words=(1 << 20) + 1)),
    (3, dict(seen=FAKE + 2)), (3, dict(lse=FAKE + 1))])
def test_tree_checks(L, code, change):  # noqa: F811
    assert L.zdmmv_attn_tree_q4_0(ctypes.byref(_cache()), ctypes.byref(_attn()), ctypes.byref(_tree(**change)), None) == code


def test_tree_words_and_nulls(L):  # noqa: F811
    c, call = _cache(), L.zdmmv_attn_tree_q4_0
    assert call(ctypes.byref(c), ctypes.byref(_attn(max_q_len=33)), ctypes.byref(_tree()), None) == 2
    assert call(ctypes.byref(c), ctypes.byref(_attn(max_q_len=33, n_tok=0)), ctypes.byref(_tree(seen_words=2)), None) == 0
    assert call(ctypes.byref(c), ctypes.byref(_attn(n_tok=0)), ctypes.byref(_tree(seen=None, seen_words=0)), None) == 0
    assert call(ctypes.byref(c), ctypes.byref(_attn()), None, None) == 1
    assert call(ctypes.byref(c), None, ctypes.byref(_tree()), None) == 1
    assert call(None, ctypes.byref(_attn()), ctypes.byref(_tree()), None) == 1


@pytest.mark.parametrize("code, change", [
    (2, dict(n_tok=-1)), (2, dict(n_q_heads=7)), (2, dict(max_q_len=0)), (2, dict(window=-1)), (2, dict(scale=float("nan"))),
    (1, dict(q=None)), (1, dict(out=None)), (3, dict(q=FAKE + 4)), (6, dict(workspace_bytes=8192, max_kv_len=100000))])
def test_tree_takes_attentions_checks(L, code, change):  # noqa: F811
    assert L.zdmmv_attn_tree_q4_0(ctypes.byref(_cache()), ctypes.byref(_attn(**change)), ctypes.byref(_tree()), None) == code


def test_binding_refuses_bad_bits():
    with pytest.raises(ValueError):
        Z._seen(torch.zeros(3, dtype=torch.int32), 3)
    with pytest.raises(ValueError):
        Z._seen(torch.zeros(2, 1, dtype=torch.int32), 3)
    with pytest.raises(ValueError):
        Z._seen(torch.zeros(3, 1, dtype=torch.int32), 3)     # a host tensor
    assert Z._seen(None, 3) == (0, 0)
