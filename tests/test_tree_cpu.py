"""The operators on drafted trees and eviction without a GPU: argument checks and structs."""
import ctypes

import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import test_block_ops_cpu as B
from tests.test_block_ops_cpu import FAKE, L, _attn, _cache, _header_fields  # noqa: F401


class _AttnTree(ctypes.Structure):
    _fields_ = [("seen", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("seen_words", ctypes.c_int32)]


class _AttnWeightsArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "q_start", "kv_len", "lse", "seen", "before", "out", "workspace", "status_dev")] + [
        ("workspace_bytes", ctypes.c_size_t)] + [(n, ctypes.c_int64) for n in ("q_stride", "before_stride", "out_stride")] + [
        (n, ctypes.c_int32) for n in ("n_tok", "n_q_heads", "max_q_len", "max_kv_len", "window", "seen_words")] + [
        (n, ctypes.c_float) for n in ("scale", "keep")]


class _KvEvictArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("kv_len", "sums", "index", "sums_out", "len_out", "status_dev")] + [
        (n, ctypes.c_int64) for n in ("sums_stride", "sums_out_stride")] + [
        (n, ctypes.c_int32) for n in ("max_kv_len", "budget", "sinks", "recent")]


class _KvAcceptArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("base", "path", "n_path", "len_out", "status_dev", "sums")] + [
        (n, ctypes.c_int64) for n in ("sums_stride", "sums_len")] + [("max_path", ctypes.c_int32)]


@pytest.mark.parametrize("name, c, packed", [
    ("zdmmv_attn_tree", _AttnTree, Z._ATTN_TREE), ("zdmmv_attn_weights_args", _AttnWeightsArgs, Z._ATTN_WEIGHTS_ARGS),
    ("zdmmv_kv_evict_args", _KvEvictArgs, Z._KV_EVICT_ARGS), ("zdmmv_kv_accept_args", _KvAcceptArgs, Z._KV_ACCEPT_ARGS)])
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


def _weights(**k):
    d = dict(q=FAKE, q_start=FAKE, kv_len=FAKE, lse=FAKE, seen=FAKE, before=FAKE, out=2 * FAKE, workspace=None, status_dev=FAKE, workspace_bytes=0, q_stride=1024,
             before_stride=100, out_stride=100, n_tok=3, n_q_heads=8, max_q_len=2, max_kv_len=100, window=0, seen_words=1, scale=0.1,
             keep=1.0)
    return _AttnWeightsArgs(**{**d, **k})


@pytest.mark.parametrize("code, change", [
    (2, dict(n_tok=-1)), (2, dict(n_q_heads=7)), (2, dict(n_q_heads=0)), (2, dict(n_q_heads=65536)), (2, dict(max_q_len=0)),
    (2, dict(max_kv_len=-1)), (2, dict(window=-1)), (2, dict(scale=float("nan"))), (2, dict(keep=float("inf"))),
    (2, dict(seen_words=0)), (2, dict(seen_words=(1 << 20) + 1)), (2, dict(max_q_len=33)), (2, dict(q_stride=1000)),
    (2, dict(out_stride=99)), (2, dict(before_stride=99)), (2, dict(before=2 * FAKE, before_stride=104)),
    (1, dict(q=None)), (1, dict(q_start=None)), (1, dict(kv_len=None)), (1, dict(lse=None)), (1, dict(out=None)),
    (3, dict(q=FAKE + 4)), (3, dict(q_stride=1026)), (3, dict(q_start=FAKE + 1)), (3, dict(kv_len=FAKE + 2)), (3, dict(lse=FAKE + 2)),
    (3, dict(seen=FAKE + 2)), (3, dict(before=FAKE + 1)), (3, dict(out=FAKE + 2)), (3, dict(status_dev=FAKE + 2)),
    (1, dict(n_tok=40, max_q_len=32)), (6, dict(n_tok=40, max_q_len=32, workspace=FAKE, workspace_bytes=4096)),
    (3, dict(workspace=FAKE + 8)), (0, dict(max_kv_len=0, q=None, out=None))])
def test_weights_checks(L, code, change):  # noqa: F811
    assert L.zdmmv_attn_weights_q4_0(ctypes.byref(_cache()), ctypes.byref(_weights(**change)), None) == code


def _evict(**k):
    d = dict(kv_len=FAKE, sums=FAKE, index=FAKE, sums_out=2 * FAKE, len_out=FAKE, status_dev=FAKE, sums_stride=100, sums_out_stride=64,
             max_kv_len=100, budget=64, sinks=4, recent=16)
    return _KvEvictArgs(**{**d, **k})


@pytest.mark.parametrize("code, change", [
    (2, dict(max_kv_len=-1)), (2, dict(max_kv_len=0x7fff0001, sums_stride=1 << 40)), (2, dict(budget=0)), (2, dict(budget=129, sums_out_stride=200)),
    (2, dict(sinks=-1)), (2, dict(recent=-1)), (2, dict(sinks=49)), (2, dict(sinks=0x7fffffff, recent=0x7fffffff)),
    (2, dict(sums_stride=99)), (2, dict(sums_out_stride=63)), (2, dict(sums_out=FAKE)),
    (1, dict(kv_len=None)), (1, dict(sums=None)), (1, dict(index=None)),
    (3, dict(kv_len=FAKE + 2)), (3, dict(sums=FAKE + 1)), (3, dict(index=FAKE + 2)), (3, dict(sums_out=FAKE + 2)), (3, dict(len_out=FAKE + 1)),
    (3, dict(status_dev=FAKE + 2))])
def test_evict_checks(L, code, change):  # noqa: F811
    assert L.zdmmv_kv_evict_q4_0(ctypes.byref(_cache()), ctypes.byref(_cache()), ctypes.byref(_evict(**change)), None) == code


@pytest.mark.parametrize("code, change", [(2, dict(n_seq=3)), (2, dict(n_kv_heads=1)), (2, dict(head_dim=64)), (2, dict(page_tokens=20)),
                                          (1, dict(pages=None)), (3, dict(pages=FAKE + 8))])
def test_evict_checks_both_caches(L, code, change):  # noqa: F811
    call = L.zdmmv_kv_evict_q4_0
    assert call(ctypes.byref(_cache()), ctypes.byref(_cache(**change)), ctypes.byref(_evict()), None) == code
    assert call(ctypes.byref(_cache(**change)), ctypes.byref(_cache()), ctypes.byref(_evict()), None) == code


def test_evict_refuses_the_cache_itself(L):  # noqa: F811
    c, again = _cache(), _cache()
    assert L.zdmmv_kv_evict_q4_0(ctypes.byref(c), ctypes.byref(again), ctypes.byref(_evict()), None) == 2


def _accept(**k):
    return _KvAcceptArgs(**{**dict(base=FAKE, path=FAKE, n_path=FAKE, len_out=FAKE, status_dev=FAKE, sums=FAKE, sums_stride=128, sums_len=100, max_path=8), **k})


@pytest.mark.parametrize("code, change", [
    (2, dict(max_path=0)), (2, dict(max_path=1025)), (2, dict(sums_stride=99)), (2, dict(sums_len=7)), (3, dict(sums=FAKE + 2)), (1, dict(base=None)), (1, dict(path=None)), (1, dict(n_path=None)),
    (3, dict(base=FAKE + 1)), (3, dict(path=FAKE + 2)), (3, dict(n_path=FAKE + 2)), (3, dict(len_out=FAKE + 2)), (3, dict(status_dev=FAKE + 2))])
def test_accept_checks(L, code, change):  # noqa: F811
    assert L.zdmmv_kv_accept_q4_0(ctypes.byref(_cache()), ctypes.byref(_accept(**change)), None) == code


def test_append_at_checks(L):  # noqa: F811
    assert L.zdmmv_kv_append_at_q4_0(ctypes.byref(_cache()), ctypes.byref(B._append()), FAKE + 2, None) == 3
    assert L.zdmmv_kv_append_at_q4_0(ctypes.byref(_cache()), ctypes.byref(B._append(n_tok=0)), FAKE, None) == 0
    assert L.zdmmv_kv_append_at_q4_0(ctypes.byref(_cache()), ctypes.byref(B._append(rot_dim=3)), FAKE, None) == 2


def test_null_structs(L):  # noqa: F811
    c = ctypes.byref(_cache())
    assert L.zdmmv_attn_weights_q4_0(c, None, None) == 1 and L.zdmmv_attn_weights_q4_0(None, ctypes.byref(_weights()), None) == 1
    assert L.zdmmv_kv_accept_q4_0(c, None, None) == 1 and L.zdmmv_kv_accept_q4_0(None, ctypes.byref(_accept()), None) == 1
    assert L.zdmmv_kv_evict_q4_0(c, c, None, None) == 1 and L.zdmmv_kv_evict_q4_0(c, None, ctypes.byref(_evict()), None) == 1
    assert L.zdmmv_kv_append_at_q4_0(c, None, FAKE, None) == 1


def test_weights_workspace(L):  # noqa: F811
    size = lambda heads, tok, new, **k: L.zdmmv_attn_weights_q4_0_workspace_bytes(ctypes.byref(_cache(**k)), heads, tok, new)  # noqa: E731
    assert size(8, 6, 6) == 0 and size(8, 100, 6) == 0 and size(8, 6, 100) == 0      # 24 columns
    assert size(8, 7, 7) > 0 and size(16, 4, 4) > 0
    assert size(7, 9, 9) == 0 and size(8, -1, 9) == 0 and size(8, 9, 0) == 0         # refused shapes
    last = 0
    for tok in (9, 10, 16, 17, 100, 101, 1000):
        assert size(8, tok, 9) >= last
        last = size(8, tok, 9)
    # blocks of 64 columns of q in two fp16 parts and 16 bytes a column: those of the rows, and one a sequence
    assert size(8, 1000, 9) == (1000 * 4 // 64 + 2) * 2 * (64 * (128 * 4 + 16) + 16)


def test_weights_waits_that_gave_up():
    """Every wait of the tall kernel that reports a fault marks its thread, and a marked thread makes the result NaN."""
    from tests.test_gave_up_waits_cpu import block, source, waits_that_report
    text = source("zdmmv_attn_weights.cu")
    assert text.count("atomicOr(a.fault") == 1
    assert ["dead = true" in b for b in waits_that_report(text)] == [True]
    kernel = block(text, text.index("attn_weights_tall_kernel(WeightArgs w)"))
    after = kernel[kernel.index("if (dead) sh_dead = 1;"):]
    assert "wait(" not in after and after.index("__syncthreads()") < after.index("if (sh_dead) sum = ")


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would run")
@pytest.mark.parametrize("head_dim", [64, 128, 256])
def test_attentions_workspace_is_one_for_trees(L, head_dim):  # noqa: F811
    """A tree's plan does with what zdmmv_attn_q4_0_workspace_bytes asks for, whatever the shape."""
    import itertools
    for n_seq, heads, group, new, most, window in itertools.product((1, 2, 7, 40, 300, 700), (1, 4, 8), (1, 4, 5, 8), (1, 3, 5, 12, 25, 64, 300),
                                                                   (1, 300, 2011, 9000, 65536), (0, 1000)):
        c = _cache(n_seq=n_seq, n_kv_heads=heads, head_dim=head_dim, max_pages=1 << 16)
        size = L.zdmmv_attn_q4_0_workspace_bytes(ctypes.byref(c), heads * group, new, most)
        args = _attn(n_q_heads=heads * group, q_stride=heads * group * head_dim, max_q_len=new, max_kv_len=most, window=window,
                     n_tok=new, workspace=FAKE if size else None, workspace_bytes=size)
        got = L.zdmmv_attn_tree_q4_0(ctypes.byref(c), ctypes.byref(args), ctypes.byref(_tree(seen_words=10)), None)
        assert got not in (1, 2, 6), (n_seq, heads, group, new, most, window, got)


def test_binding_refuses_bad_sums():
    """[n_seq][n_kv_heads][tokens] with kv heads evenly apart; views of a wider buffer pass."""
    class Cache:
        n_seq, n_kv_heads = 2, 3

    class Tensor:  # a CUDA tensor's looks
        dtype, is_cuda = torch.float32, True

        def __init__(self, t):
            self.shape, self.stride, self.data_ptr = t.shape, t.stride, lambda: 256
    wide = torch.zeros(2, 3, 50)
    assert Z._per_head(Tensor(wide), Cache, 50, "x") == (256, 50)
    assert Z._per_head(Tensor(wide[:, :, :40]), Cache, 40, "x") == (256, 50)
    for bad in (wide[:1], wide[:, :2], wide[:, :, :30], torch.zeros(2, 4, 50)[:, :3], wide.transpose(0, 1), torch.zeros(2, 3, 100)[:, :, ::2],
                wide[0], torch.zeros(150)):
        with pytest.raises(ValueError):
            Z._per_head(Tensor(bad), Cache, 40, "x")
    Cache.n_seq, Cache.n_kv_heads = 1, 1
    assert Z._per_head(Tensor(torch.zeros(1, 1, 7)), Cache, 7, "x") == (256, 7)
    Cache.n_seq = 2
    assert Z._per_head(Tensor(torch.zeros(2, 9, 7)[:, :1]), Cache, 7, "x") == (256, 63)
    with pytest.raises(ValueError):
        Z._per_head(torch.zeros(2, 1, 7), Cache, 7, "x")  # a host tensor
