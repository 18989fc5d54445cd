"""The attention's workspace without a GPU: its size holds for every call within the bounds that it was asked for."""
import ctypes
import itertools

import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests.test_block_ops_cpu import _attn, _cache

SEQS = [1, 2, 3, 5, 8, 13, 20, 25, 26, 38, 40, 48, 50, 64, 77, 100, 128, 200, 257, 300, 400, 512]
LENGTHS = [0, 1, 16, 17, 255, 256, 257, 300, 600, 1000, 1500, 2049, 2060, 2064, 2100, 2304, 2600, 3000, 4100, 4120, 6000, 8192,
           12000, 16384, 20000, 40000, 131072, 1 << 20]


def sizer(n_seq, kv_heads, head_dim, heads):
    c = _cache(n_seq=n_seq, n_kv_heads=kv_heads, head_dim=head_dim, max_pages=1 << 16)
    return lambda new, most: Z.lib().zdmmv_attn_q4_0_workspace_bytes(ctypes.byref(c), heads, new, most)


@pytest.mark.parametrize("head_dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kv_heads", [1, 4, 8, 16])
def test_a_longer_bound_never_needs_less(kv_heads, head_dim):
    """A window shortens what a call works on, and lengths below the bound are what it is for."""
    for n_seq, group, new in itertools.product(SEQS, (1, 4, 5, 8), (1, 2, 4, 9, 40, 300)):
        size = sizer(n_seq, kv_heads, head_dim, kv_heads * group)
        last = 0
        for most in LENGTHS:
            now = size(new, most)
            assert now >= last, (n_seq, group, new, most)
            last = now


def test_the_windowed_call_of_48_sequences():
    """Stretches over all steps at 16384 tokens, two splits of 384 items at the 2048 that its window sees: 768 parts of four
    columns of 128 sums, a maximum and a sum of p."""
    size = sizer(48, 8, 128, 32)
    assert size(1, 16384) >= size(1, 2100) >= 8192 + 768 * 4 * 130 * 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="what is not refused would run")
def test_a_call_checks_what_it_launches():
    c = _cache(n_seq=48, n_kv_heads=8, max_pages=1 << 16)
    need = 8192 + 768 * 4 * 130 * 4
    call = lambda **k: Z.lib().zdmmv_attn_q4_0(ctypes.byref(c), ctypes.byref(_attn(  # noqa: E731
        n_q_heads=32, q_stride=4096, max_q_len=1, n_tok=48, window=2048, max_kv_len=16384, **k)), None)
    assert call(workspace_bytes=need - 1) == 6
    assert call(workspace=None) == 1
    assert call(workspace_bytes=need) not in (1, 6)


@pytest.mark.parametrize("head_dim", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("kv_heads", [1, 4, 8, 16])
def test_more_new_tokens_never_need_less(kv_heads, head_dim):
    """A workspace made for a prompt's chunk is one for decoding."""
    for n_seq, group, most in itertools.product(SEQS, (1, 3, 4, 5, 8), LENGTHS[::3]):
        size = sizer(n_seq, kv_heads, head_dim, kv_heads * group)
        last = 0
        for new in (1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 13, 16, 17, 24, 33, 40, 65, 100, 128, 129, 200, 300, 600, 2000):
            now = size(new, most)
            assert now >= last, (n_seq, group, new, most)
            last = now


def test_the_workspace_of_300_sequences_serves_eight_new_tokens_and_one():
    """Eight new tokens of four heads make more items than there are counters, which are not split; one is walked."""
    size = sizer(300, 8, 128, 32)
    assert size(8, 4096) >= size(1, 4096) >= 8192 + 608 * 4 * 130 * 4


def test_sizes_stay_within_reason():
    """Twice as many parts as run at once, or four times as many CTAs of 128 columns as the device has SMs."""
    for head_dim, kv_heads, n_seq, new in itertools.product((64, 128, 256), (1, 8), (1, 40, 300), (1, 8, 4096)):
        size = sizer(n_seq, kv_heads, head_dim, 4 * kv_heads)(new, 1 << 20)
        assert size <= 8192 + 4 * 152 * 128 * (head_dim + 2) * 4
