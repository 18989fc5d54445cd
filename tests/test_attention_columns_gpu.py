"""Attention of more than 16 columns (new tokens x query heads of a kv head) on the GPU against the plain restatement in
64 bits (tests/block_ref.py): the form whose products run on tcgen05 for heads of up to 128 dimensions.

Bounds. k = d (n - 8) is the sum of two fp16 numbers exactly, q of two to 2^-22. A score leaves out the product of the two
lower parts (2^-22 of its terms' sizes) and adds up to 24 times with truncation (2^-23 of at most P each, P = scale *
sum |q_e| max|k_block|): its error is below 2^-18 P, p's relative error and so the result's twice that. A tile's sum of
p v adds 24 times too, and tiles (up to 64) are added in fp32: below 2^-17 of sum p max|v_block|.
"""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests.test_block_ops_gpu import dev, random_cache

pytestmark = pytest.mark.gpu


def check(out, q, q_start, lens, table, pages, page, heads, dim, scale, window):
    k, v = R.values(pages, page, heads, dim)
    want, tp, tv = R.attention(q, q_start, lens, table, k, v, page, scale, window)
    got = out.double().cpu().numpy()
    tol = tv * (2 * 2.0 ** -18 * tp + 2.0 ** -17)[..., None]
    assert np.isfinite(got).all()
    bad = np.abs(got - want) - tol
    assert (bad <= 0).all(), (bad.max(), np.abs(got - want).max(), np.unravel_index(bad.argmax(), bad.shape))


def run(seed, lens, new, page, heads, group, dim, window=0, scale=None, sharp=1.5, scales=None):
    rng = np.random.default_rng(seed)
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    if scales is not None:
        scales(rng, pages.reshape(-1, heads, page // 16, 18 * dim), table)
        cache.pages.copy_(dev(pages))
    q_start = np.concatenate(([0], np.cumsum(new))).astype(np.int32)
    q = (sharp * rng.standard_normal((q_start[-1], heads * group, dim))).astype(np.float32)
    scale = dim ** -0.5 if scale is None else scale
    args = (cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), max(new), max(lens))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full(q.shape, float("nan"), device="cuda")
    Z.attn_q4_0(*args, scale=scale, window=window, out=out, status=status)
    assert status.item() == 0
    check(out, q, q_start, lens, table, pages, page, heads, dim, scale, window)
    assert torch.equal(Z.attn_q4_0(*args, scale=scale, window=window), out)  # the same bits again


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("heads, group, lens, new, window", [
    (1, 17, [1], [1], 0), (2, 4, [16, 127], [5, 5], 0), (2, 5, [128, 0, 129], [4, 1, 5], 0), (1, 1, [127], [127], 0),
    (1, 1, [400], [128], 0), (1, 1, [400], [129], 50), (2, 2, [901], [65], 0), (1, 8, [255, 3000], [3, 8], 700),
    (1, 32, [1025], [1], 1), (3, 8, [20, 5], [24, 9], 0)])   # the last: more new tokens than the cache holds, empty rows
def test_columns(dim, heads, group, lens, new, window):
    run(dim + sum(lens) + group, lens, new, 48, heads, group, dim, window=window)


@pytest.mark.parametrize("page, lens, new", [(16, [8000], [16]), (128, [5003, 17, 2900], [8, 8, 8])])
def test_many_parts(page, lens, new):
    run(sum(lens), lens, new, page, 1, 4, 128)


@pytest.mark.parametrize("sharp, scale", [(30.0, None), (0.0, None), (1.0, 0.0), (1.0, -0.3), (1e-20, 1.0), (1e4, 1e-3)])
def test_scores_of_any_size(sharp, scale):
    run(5, [777, 60], [20, 2], 16, 2, 4, 128, scale=scale, sharp=sharp)


@pytest.mark.parametrize("dim", [64, 96, 128])
@pytest.mark.parametrize("which", ["k", "v", "both"])
def test_scales_whose_values_are_no_fp16_numbers(dim, which):
    """Scales of 2^13 and more (8 times them is past fp16's range) in some of a sequence's tokens."""
    def scales(rng, t, table):
        for page in table[0][3:5].tolist() + table[0][17:18].tolist():
            for at in [16] * (which != "v") + [17] * (which != "k"):
                sc = np.exp2(rng.uniform(10, 15.9, (t.shape[1], t.shape[2], dim // 2))) * rng.choice([-1, 1], (t.shape[1], t.shape[2], dim // 2))
                t[page, :, :, at * dim:(at + 1) * dim] = sc.astype(np.float16).view(np.uint8)
    run(dim + len(which), [600], [9], 32, 2, 4, dim, scale=dim ** -0.5 if which == "v" else 1e-5, scales=scales)


def test_bad_sequences():
    rng = np.random.default_rng(7)
    page, heads, group, dim, lens = 16, 2, 4, 128, [200, 200, 200]
    cache, pages, table = random_cache(rng, lens, page, heads, dim, spare=0)
    bad = table.copy()
    bad[1, 9] = 1 << 20
    cache.page_table.copy_(dev(bad))
    q = rng.standard_normal((24, heads * group, dim)).astype(np.float32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = Z.attn_q4_0(cache, dev(q), dev(np.array([0, 8, 16, 24], np.int32)), dev(np.array([200, 200, -1], np.int32)), 8, 208, status=status)
    assert status.item() == 1 and out[8:].isnan().all()
    check(out[:8], q[:8], [0, 8], lens[:1], table[:1], pages, page, heads, dim, dim ** -0.5, 0)
