"""The example's layer (examples/attention_layer.py), stage by stage: each stage against its reference on the kernels' own
input to it, for a prompt's tokens and for decode steps of several sequences."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from gguf_block_quant_gb300 import zdmmv as Z
from tests import block_ref as R
from tests.test_block_ops_gpu import U, check_attention

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def check_norm(xq, s, w, eps):
    """The blocks of one norm against the definition in 64 bits (bounds: tests/test_block_ops_gpu.py)."""
    b = xq.cpu().numpy().reshape(-1, 34)
    d = np.ascontiguousarray(b[:, :2]).view(np.float16)[:, 0].astype(np.float64)
    q = b[:, 2:].view(np.int8).astype(np.float64)
    s = s.double().cpu().numpy()
    want = (s / np.sqrt((s * s).mean(1, keepdims=True) + eps) * w.double().cpu().numpy()).reshape(-1, 32)
    step, e = np.abs(want).max(1) / 127, 100 * U
    assert np.all(np.abs(d - step) <= step * (2.0 ** -11 + e) + 2.0 ** -25)
    assert np.all(np.abs(q - want / step[:, None]) <= 0.5 + 254 * e)


def check_step(layer, r, x, residual, seq, pos, q_start, kv_len):
    c, n = layer.cfg, x.shape[0]
    s = x if residual is None else x + residual
    assert torch.equal(r["sum"], s)
    check_norm(r["xq"], s, layer.norm1, c.eps)
    y, e = oracle.dmmv_batched(Z.Q4_0, layer.w_qkv.cpu().numpy(), layer.qkv_rows, c.hidden, r["xq"].cpu().numpy(), n)
    ok, worst = oracle.within_tolerance(r["qkv"].double().cpu().numpy().reshape(n, -1), y, e)
    assert ok, worst
    rows = r["qkv"].cpu().numpy().reshape(n, -1, c.head_dim)
    turned = R.rotate(rows[:, :c.heads + c.kv_heads], layer.rope.cpu().numpy(), pos, True)
    assert np.array_equal(r["q"].cpu().numpy(), turned[:, :c.heads])
    pages = layer.cache.pages.cpu().numpy()
    table = layer.cache.page_table.cpu().numpy()
    kc, vc, kd, vd = R.unpack(pages, c.page_tokens, c.kv_heads, c.head_dim)
    for want, code, scale in ((turned[:, c.heads:], kc, kd), (rows[:, c.heads + c.kv_heads:], vc, vd)):
        wc, wd = R.quantize_q4(want)
        page, at = table[seq, pos // c.page_tokens], pos % c.page_tokens
        assert np.array_equal(code[page, :, at], wc - 8) and np.array_equal(scale[page, :, at], wd)
    check_attention(r["att"], r["q"].cpu().numpy(), q_start, kv_len, table, pages, c.page_tokens, c.kv_heads, c.head_dim)
    y, e = oracle.dmmv_batched(Z.Q4_0, layer.w_out.cpu().numpy(), c.hidden, c.heads * c.head_dim,
                               oracle.quantize_q8_0(r["att"].cpu().numpy().reshape(n, -1)), n)
    ok, worst = oracle.within_tolerance(r["out"].double().cpu().numpy(), y, e)
    assert ok, worst
    assert torch.equal(r["sum2"], r["out"] + s)
    check_norm(r["xq2"], r["sum2"], layer.norm2, c.eps)


def test_prompt_then_decode():
    from attention_layer import AttentionLayer, Config
    cfg = Config(hidden=1024, heads=8, kv_heads=2, head_dim=128, page_tokens=32, max_len=256)
    lens = [3, 17, 40]
    layer = AttentionLayer(cfg, len(lens))
    g = torch.Generator("cuda").manual_seed(11)
    i32 = lambda v: torch.tensor(np.asarray(v, np.int32), device="cuda")  # noqa: E731
    for s, n in enumerate(lens):
        for p in range(0, n, 8):
            m = min(8, n - p)
            x = torch.randn(m, cfg.hidden, device="cuda", generator=g)
            seq, pos = np.full(m, s), np.arange(p, p + m)
            q_start = np.array([0] * (s + 1) + [m] * (len(lens) - s))
            kv_len = np.array([p + m if t == s else 0 for t in range(len(lens))])
            r = layer.step(x, None, i32(seq), i32(pos), i32(q_start), i32(kv_len), m)
            check_step(layer, r, x, None, seq, pos, q_start, kv_len)
    for step in range(2):
        x, res = (torch.randn(3, cfg.hidden, device="cuda", generator=g) for _ in range(2))
        seq, pos = np.arange(3), np.array(lens) + step
        r = layer.step(x, res, i32(seq), i32(pos), i32(np.arange(4)), i32(pos + 1), 1)
        check_step(layer, r, x, res, seq, pos, np.arange(4), pos + 1)
    assert Z.device_status() == 0


def test_the_example_runs(capsys):
    import attention_layer
    attention_layer.main(steps=8)
    assert "us a step" in capsys.readouterr().out
