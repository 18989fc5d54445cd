"""The attention's workspace on the GPU: nothing behind it (nor behind the result) is written, in the shapes where the call's
plan is another than the one of its longest sequence."""
import numpy as np
import pytest
import torch

from gguf_block_quant_gb300 import zdmmv as Z
from tests.test_block_ops_gpu import check_attention, dev, random_cache, ragged

pytestmark = pytest.mark.gpu

GUARD = 4 << 20


def guarded(n, value=0xA5):
    """n bytes (a multiple of 16) with others behind them."""
    buf = torch.full((n + GUARD,), value, dtype=torch.uint8, device="cuda")
    return buf[:n], buf[n:]


@pytest.mark.parametrize("n_seq, heads, group, dim, new, window, longest, bound", [
    (48, 8, 4, 128, 1, 2048, 2300, 16384), (40, 8, 4, 128, 1, 2048, 2300, 8192), (13, 16, 1, 64, 1, 4096, 4400, 65536),
    (22, 8, 4, 128, 4, 2048, 2300, 16384), (22, 8, 2, 256, 1, 2048, 2300, 16384)])
def test_windows_over_many_sequences(n_seq, heads, group, dim, new, window, longest, bound):
    rng = np.random.default_rng(n_seq + dim)
    page = 64
    lens = [max(n, new) for n in ragged(rng, n_seq, longest)]
    cache, pages, table = random_cache(rng, lens, page, heads, dim)
    q_start = np.arange(n_seq + 1, dtype=np.int32) * new
    q = (1.5 * rng.standard_normal((n_seq * new, heads * group, dim))).astype(np.float32)
    # the longest that the call allows is further than these sequences are: their table has room for it
    wide = np.full((n_seq, -(-bound // page)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    cache = Z.KVCache(cache.pages, page, heads, dim, dev(wide))
    size = Z.attn_q4_0_workspace_bytes(cache, heads * group, new, bound)
    ws, behind = guarded(size)
    ws[:8192] = 0
    room, after = guarded(q.nbytes)
    out = room.view(torch.float32).view(q.shape)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = (cache, dev(q), dev(q_start), dev(np.array(lens, np.int32)), new, bound)
    Z.attn_q4_0(*args, window=window, out=out, workspace=ws, status=status)
    assert status.item() == 0
    assert (behind == 0xA5).all() and (after == 0xA5).all() and not ws[:8192].any()
    assert torch.equal(Z.attn_q4_0(*args, window=window), out)      # a workspace of the call's own
    whole = np.ascontiguousarray(pages).reshape(-1, Z.kv_page_bytes(page, heads, dim))
    for s in range(n_seq):
        held = -(-lens[s] // page)
        rows = slice(s * new, (s + 1) * new)
        check_attention(out[rows], q[rows], [0, new], lens[s:s + 1], np.arange(held)[None], whole[table[s, :held]], page, heads,
                        dim, window=window)


def test_a_prompts_workspace_serves_decoding():
    """One workspace for up to eight new tokens of 300 sequences, then calls of eight, three and one new tokens on it."""
    rng = np.random.default_rng(300)
    n_seq, heads, group, dim, page, bound = 300, 8, 4, 128, 64, 4096
    lens = [max(8, n) for n in ragged(rng, n_seq, 700)]
    cache, _, table = random_cache(rng, lens, page, heads, dim)
    wide = np.full((n_seq, bound // page), -1, np.int32)
    wide[:, :table.shape[1]] = table
    cache = Z.KVCache(cache.pages, page, heads, dim, dev(wide))
    size = Z.attn_q4_0_workspace_bytes(cache, heads * group, 8, bound)
    ws, behind = guarded(size)
    ws[:8192] = 0
    kv_len = dev(np.array(lens, np.int32))
    for new in (8, 1, 3, 1):
        q_start = dev(np.arange(n_seq + 1, dtype=np.int32) * new)
        q = torch.randn(n_seq * new, heads * group, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(new))
        out = Z.attn_q4_0(cache, q, q_start, kv_len, new, bound, workspace=ws)
        assert torch.equal(Z.attn_q4_0(cache, q, q_start, kv_len, new, bound), out)
        assert (behind == 0xA5).all() and not ws[:8192].any()
