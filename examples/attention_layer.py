"""The attention half of a decode layer on the library's own operators, step by step:

    norm     s = x + residual, Q8_0 blocks of norm(s)          add_rmsnorm_q8_0
    qkv      the joint projection of the blocks                dmmv_batched (Q4_0 weights)
    append   q and k rotated, k and v into the paged cache     kv_append_q4_0
    attend   softmax(q k^T) v over the cache                   attn_q4_0
    out      the output projection                             dmmv_f32 (quantizes its input)
    norm     s' = s + out, Q8_0 blocks for the FFN             add_rmsnorm_q8_0

``python examples/attention_layer.py`` decodes a few steps of three sequences of different lengths (a call takes up to
8 tokens, as the batched DMMV does) with synthetic weights, first their prompts, then token by token, the decode step
replayed as a CUDA graph, and prints the time of a step.
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gguf_block_quant_gb300 import synth, zdmmv as Z  # noqa: E402


@dataclass
class Config:
    hidden: int = 2048
    heads: int = 16
    kv_heads: int = 4
    head_dim: int = 128
    page_tokens: int = 64
    max_len: int = 4096
    eps: float = 1e-6
    seed: int = 0


class AttentionLayer:
    def __init__(self, cfg: Config, n_seq: int):
        c = self.cfg = cfg
        self.n_seq = n_seq
        self.qkv_rows = (c.heads + 2 * c.kv_heads) * c.head_dim
        g = torch.Generator("cuda").manual_seed(c.seed)
        self.w_qkv = torch.from_numpy(synth.weight_blocks(Z.Q4_0, self.qkv_rows, c.hidden, seed=c.seed)).cuda()
        self.w_out = torch.from_numpy(synth.weight_blocks(Z.Q4_0, c.hidden, c.heads * c.head_dim, seed=c.seed + 1)).cuda()
        self.norm1, self.norm2 = (1 + 0.1 * torch.randn(c.hidden, device="cuda", generator=g) for _ in range(2))
        angle = np.arange(c.max_len)[:, None] * 10000.0 ** (-np.arange(c.head_dim // 2) * 2.0 / c.head_dim)
        self.rope = torch.from_numpy(np.concatenate((np.cos(angle), np.sin(angle)), 1).astype(np.float32)).cuda()
        # every sequence has its pages from the start; an engine would hand them out as the sequences grow
        per_seq = -(-c.max_len // c.page_tokens)
        pages = torch.zeros(n_seq * per_seq * Z.kv_page_bytes(c.page_tokens, c.kv_heads, c.head_dim), dtype=torch.uint8, device="cuda")
        table = torch.randperm(n_seq * per_seq, generator=g, device="cuda").to(torch.int32).view(n_seq, per_seq)
        self.cache = Z.KVCache(pages, c.page_tokens, c.kv_heads, c.head_dim, table)
        self.workspace = Z.attn_q4_0_workspace(self.cache, c.heads, Z.MAX_BATCH, c.max_len)

    def step(self, x, residual, seq, pos, q_start, kv_len, max_new: int):
        """One call's tokens (1 to 8 rows of x, fp32) through the layer: seq and pos [tokens], q_start [sequences + 1],
        kv_len [sequences] (the new tokens included). Returns every intermediate result by name."""
        c, n = self.cfg, x.shape[0]
        s = torch.empty_like(x)
        xq = Z.add_rmsnorm_q8_0(x, self.norm1, c.eps, residual=residual, out=s)
        qkv = Z.dmmv_batched(Z.Q4_0, self.w_qkv, self.qkv_rows, c.hidden, xq, n)
        q, k, v = qkv.split((c.heads * c.head_dim, c.kv_heads * c.head_dim, c.kv_heads * c.head_dim), 1)
        q = Z.kv_append_q4_0(self.cache, k, v, seq, pos, q=q, rope=self.rope, rope_style=Z.ROPE_HALVES)
        att = Z.attn_q4_0(self.cache, q, q_start, kv_len, max_new, c.max_len, workspace=self.workspace)
        out = Z.dmmv_f32(Z.Q4_0, self.w_out, c.hidden, c.heads * c.head_dim, att.view(n, -1), batch=n).view(n, -1)
        s2 = torch.empty_like(x)
        xq2 = Z.add_rmsnorm_q8_0(out, self.norm2, c.eps, residual=s, out=s2)
        return {"sum": s, "xq": xq, "qkv": qkv, "q": q, "att": att, "out": out, "sum2": s2, "xq2": xq2}


def main(steps: int = 32) -> None:
    cfg = Config()
    lens = [5, 700, 1900]
    layer = AttentionLayer(cfg, len(lens))
    g = torch.Generator("cuda").manual_seed(7)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    # the prompts, eight tokens of one sequence at a time
    for s, n in enumerate(lens):
        for p in range(0, n, Z.MAX_BATCH):
            m = min(Z.MAX_BATCH, n - p)
            starts = [0] * (s + 1) + [m] * (len(lens) - s)
            layer.step(torch.randn(m, cfg.hidden, device="cuda", generator=g), None, i32([s] * m), i32(range(p, p + m)),
                       i32(starts), i32([p + m if t == s else 0 for t in range(len(lens))]), m)
    # one token of each sequence a step, as a graph whose positions advance on the device
    x = torch.randn(len(lens), cfg.hidden, device="cuda", generator=g)
    seq, pos, kv_len = i32(range(len(lens))), i32(lens), i32([n + 1 for n in lens])
    q_start = i32(range(len(lens) + 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, None, seq, pos, q_start, kv_len, 1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r = layer.step(x, None, seq, pos, q_start, kv_len, 1)
            pos.add_(1)
            kv_len.add_(1)
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(side)
        for _ in range(steps):
            graph.replay()
        e1.record(side)
    torch.cuda.synchronize()
    assert torch.isfinite(r["sum2"]).all() and Z.device_status() == 0
    print(f"{len(lens)} sequences of {[n + steps for n in lens]} tokens: {e0.elapsed_time(e1) / steps * 1e3:.1f} us a step of one layer")


if __name__ == "__main__":
    main()
