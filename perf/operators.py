"""The decode block's operators around the DMMV, as cases to measure.

Three operators of a transformer layer's attention half, in their plain form (elementary torch operations in fp32) and
through the library:

  norm    s = x + r, y = s / sqrt(mean(s^2) + eps) * w, quantized to Q8_0 blocks: what feeds a projection's DMMV
  append  the position rotation of q and k, k and v quantized to Q4_0 blocks and put into a paged cache
  attn    softmax(q k^T scale) v over the paged 4-bit cache: one token a sequence, a few (drafted tokens being
          verified), or a prompt's chunk; causal, ragged lengths, an optional window

The cache is laid out in tiles of 16 tokens of one head, 18 bytes for each of the head's dimensions: the codes of K,
the codes of V, the scales of K, the scales of V. `code_index` and `scale_index` say where a token's values lie in a
tile.
"""
import math
import random

import numpy as np
import torch

own = False

QK = 32          # values of a quantized block
SLAB = 16        # tokens of a cache tile
EPS = 1e-6
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode token through a small model's norm: latency alone
        {"name": "norm 1x2048", "op": "norm", "rows": 1, "cols": 2048},
        # the largest batched DMMV call's activations
        {"name": "norm 8x4096", "op": "norm", "rows": 8, "cols": 4096},
        # a width of an odd number of blocks, an odd number of rows
        {"name": "norm 777x1312", "op": "norm", "rows": 777, "cols": 1312},
        # a prompt's activations: bound by memory
        {"name": "norm 4096x4096", "op": "norm", "rows": 4096, "cols": 4096},
        # one decode token, wide heads of which a quarter is rotated
        {"name": "append 1 token d256", "op": "append", "seqs": 1, "tokens": 1, "heads": 16, "kv_heads": 2, "dim": 256,
         "page": 64, "rot": 64, "halves": True, "start": 500},
        # one token of each of 48 sequences, small pages, rotation of neighbouring pairs
        {"name": "append 48 seqs", "op": "append", "seqs": 48, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "rot": 128, "halves": False, "start": 1000},
        # a prompt of an odd length at once
        {"name": "append prompt 4093", "op": "append", "seqs": 1, "tokens": 4093, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "rot": 128, "halves": True, "start": 0},
        # one sequence early in its life: latency alone
        {"name": "attn 1x777 d256", "op": "attn", "seqs": 1, "tokens": 1, "heads": 16, "kv_heads": 2, "dim": 256,
         "page": 64, "longest": 777, "shortest": 777, "window": 0},
        # one sequence with a very long context: few rows, the work split over the length
        {"name": "attn 1x130975", "op": "attn", "seqs": 1, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "longest": 130975, "shortest": 130975, "window": 0},
        # a serving batch of ragged lengths (one of them without any token yet) on small pages
        {"name": "attn 64 ragged 16384", "op": "attn", "seqs": 64, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "longest": 16384, "shortest": 0, "window": 0},
        # drafted tokens being verified, a head of its own for every query head, a sliding window
        {"name": "attn 8x5 window", "op": "attn", "seqs": 8, "tokens": 5, "heads": 16, "kv_heads": 16, "dim": 64,
         "page": 32, "longest": 8191, "shortest": 3, "window": 4096},
        # a chunk of a prompt over what came before it
        {"name": "attn chunk 256x8192", "op": "attn", "seqs": 1, "tokens": 256, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "longest": 8192, "shortest": 8192, "window": 0},
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n in (96, 3072) else n  # one width that these cases do without, in values and in blocks


def draw(rng):
    op = rng.choice(["norm", "append", "attn", "attn"])
    if op == "norm":
        cols = QK * _log(rng, 8, 256)
        return {"op": op, "rows": _log(rng, 1, max(1, min(8192, (1 << 24) // cols))), "cols": cols}
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    if (heads + 2 * kv_heads) * dim == 3072:
        heads += kv_heads
    shape = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128])}
    if op == "append":
        seqs = _log(rng, 1, 64)
        tokens = _log(rng, 1, max(1, min(4096, (1 << 24) // (seqs * (heads + 2 * kv_heads) * dim))))
        return {**shape, "seqs": seqs, "tokens": tokens, "rot": rng.choice([dim, dim, dim // 2]),
                "halves": rng.random() < 0.5, "start": _log(rng, 1, 3000) - 1}
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    seqs, tokens = {"decode": (_log(rng, 1, 64), 1), "verify": (_log(rng, 1, 16), rng.randint(2, 8)),
                    "chunk": (rng.randint(1, 2), _log(rng, 9, 200))}[kind]
    most = {"decode": 8 * 128 * (1 << 20), "verify": 8 * 128 * (1 << 18), "chunk": 8 * 128 * 6000}[kind]
    longest = _log(rng, 20, max(21, min(131072, most // (seqs * kv_heads * dim * (heads // kv_heads + 3) // 4))))
    longest = max(longest, tokens)
    return {**shape, "seqs": seqs, "tokens": tokens, "longest": longest,
            "shortest": longest if seqs == 1 else longest // rng.choice([2, 8, 50]),
            "window": rng.choice([0, 0, 0, max(1, longest // 3)])}


def lengths(case):
    """Tokens of each sequence's context, the new ones among them: log-spread, the longest and the shortest there."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    rng = random.Random(1009 * n + hi)
    mid = [_log(rng, max(lo, hi // 16, 1), hi) for _ in range(n - 2)]
    return [hi] + mid + [lo]


# ------------------------------------------------------------------ the cache's layout
def vec_words(dim):
    """Words that a lane of a tile holds side by side."""
    nb = dim // QK
    return 4 if nb % 4 == 0 else 2 if nb % 2 == 0 else 1


def code_index(dim, device):
    """(K, V) nibble numbers in a tile's K and V codes, [SLAB][dim] each: byte n // 2, the low nibble where n is even."""
    nb, vw = dim // QK, vec_words(dim)
    r = torch.arange(SLAB, device=device)[:, None]
    e = torch.arange(dim, device=device)[None, :]
    b = e // QK
    lane = (r % 8) * 4 + (e % QK) // 8
    k = ((((r // 8) * (nb // vw) + b // vw) * 32 + lane) * vw + b % vw) * 8 + e % 8
    lane = ((e % QK) // 4) * 4 + (r % 8) // 2
    v = ((((r // 8) * (nb // vw) + b // vw) * 32 + lane) * vw + b % vw) * 8 + (r % 2) * 4 + e % 4
    return k, v


def scale_index(dim, device):
    """fp16 numbers in a tile's K (or V) scales, [SLAB][dim / QK]."""
    nb = dim // QK
    r = torch.arange(SLAB, device=device)[:, None]
    return ((r // 2) * nb + torch.arange(nb, device=device)[None, :]) * 2 + r % 2


def tile_values(tiles, dim):
    """fp32 K and V, [..., SLAB, dim] each, of tiles of bytes [..., 18 dim]."""
    out = []
    scales = tiles[..., 16 * dim:].contiguous().view(torch.float16)
    at = scale_index(dim, tiles.device)
    for which, n in enumerate(code_index(dim, tiles.device)):
        codes = tiles[..., 8 * dim * which:8 * dim * (which + 1)]
        nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
        d = scales[..., which * dim // 2:(which + 1) * dim // 2][..., at].float()
        q = nib[..., n].float() - 8.0
        out.append((q.unflatten(-1, (dim // QK, QK)) * d[..., None]).flatten(-2))
    return out


def rope_table(n, rot, device):
    """fp32 [n][rot]: the cosines of the rot / 2 angles of each position, then the sines."""
    freq = ROPE_BASE ** (-torch.arange(rot // 2, dtype=torch.float64, device=device) * 2 / rot)
    angle = torch.arange(n, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat((angle.cos(), angle.sin()), 1).float()


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "norm":
        rows, cols = case["rows"], case["cols"]
        s["x"], s["r"] = 3.0 * normal(rows, cols), normal(rows, cols)
        s["w"] = 1.0 + 0.1 * normal(cols)
        if own:
            s["out"] = torch.empty(rows, cols, device="cuda")
            s["xq"] = torch.empty(rows * cols // QK * 34, dtype=torch.uint8, device="cuda")
            s["y"] = torch.empty(rows, cols, dtype=torch.float16, device="cuda")
        return s
    hq, hk, dim, page, n_seq, n = (case[k] for k in ("heads", "kv_heads", "dim", "page", "seqs", "tokens"))
    lens = lengths(case) if case["op"] == "attn" else [case["start"] + n] * n_seq
    each = max(1, -(-max(lens) // page))
    held = [max(1, -(-t // page)) for t in lens]
    n_pages = sum(held)
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32).tolist()
    table = np.zeros((n_seq, each), dtype=np.int32)
    for i, h in enumerate(held):
        table[i, :h] = [order.pop() for _ in range(h)]
    s["table"] = torch.from_numpy(table).cuda()
    page_bytes = hk * page // SLAB * 18 * dim
    if case["op"] == "append":
        # the rows of a joint projection's output, as a decode step has them
        s["qkv"] = normal(n_seq * n, (hq + 2 * hk) * dim)
        s["seq"] = torch.arange(n_seq, device="cuda", dtype=torch.int32).repeat_interleave(n)
        s["pos"] = (case["start"] + torch.arange(n, device="cuda", dtype=torch.int32)).repeat(n_seq)
        s["rope"] = rope_table(case["start"] + n, case["rot"], "cuda")
        if own:
            s["pages"] = torch.zeros(n_pages * page_bytes, dtype=torch.uint8, device="cuda")
            s["q_out"] = torch.empty(n_seq * n, hq, dim, device="cuda")
            s["k_val"], s["v_val"] = (torch.empty(n_seq * n, hk, dim, dtype=torch.float16, device="cuda") for _ in range(2))
    else:
        new = [min(n, t) if t else 1 for t in lens]
        s["q"] = 2.0 * normal(sum(new), hq, dim)
        s["new"], s["max_new"], s["max_len"] = new, max(new), max(lens)
        s["q_start"] = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device="cuda")
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["pages"] = torch.randint(0, 256, (n_pages * page_bytes,), generator=g, device="cuda", dtype=torch.uint8)
        tiles = s["pages"].view(-1, 18 * dim)
        d = torch.rand(tiles.shape[0], dim, generator=g, device="cuda") * 0.2 + 0.1
        d = torch.where(torch.rand(d.shape, generator=g, device="cuda") < 0.5, -d, d).half()
        tiles[:, 16 * dim:] = d.view(torch.uint8)
        if own:
            s["out"] = torch.empty(sum(new), hq, dim, device="cuda")
    if own:
        from gguf_block_quant_gb300 import zdmmv as Z
        s["cache"] = Z.KVCache(s["pages"], page, hk, dim, s["table"])
        if case["op"] == "attn":
            s["workspace"] = Z.attn_q4_0_workspace(s["cache"], hq, s["max_new"], s["max_len"])
    return s


# ------------------------------------------------------------------ the operators
def run(s):
    c = s["case"]
    if own:
        return {"norm": _own_norm, "append": _own_append, "attn": _own_attn}[c["op"]](s)
    return {"norm": _norm, "append": _append, "attn": _attn}[c["op"]](s)


def _own_norm(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    Z.add_rmsnorm_q8_0(s["x"], s["w"], EPS, residual=s["r"], out=s["out"], xq=s["xq"], y=s["y"])
    return {"sum": s["out"], "y": s["y"]}


def _own_append(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    c, qkv = s["case"], s["qkv"]
    hq, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    q, k, v = qkv[:, :hq * dim], qkv[:, hq * dim:(hq + hk) * dim], qkv[:, (hq + hk) * dim:]
    Z.kv_append_q4_0(s["cache"], k, v, s["seq"], s["pos"], q=q, q_out=s["q_out"], rope=s["rope"],
                     rope_style=Z.ROPE_HALVES if c["halves"] else Z.ROPE_PAIRS, k_val=s["k_val"], v_val=s["v_val"])
    return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}


def _own_attn(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    return Z.attn_q4_0(s["cache"], s["q"], s["q_start"], s["kv_len"], s["max_new"], s["max_len"],
                       window=s["case"]["window"], out=s["out"], workspace=s["workspace"])


def _away(v):
    """Rounds to whole numbers, halves away from zero."""
    t = torch.trunc(v)
    return t + torch.where((v - t).abs() >= 0.5, torch.sign(v), torch.zeros_like(v))


def _norm(s):
    x = s["x"] + s["r"]
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    y = (x * rstd * s["w"]).unflatten(-1, (-1, QK))
    d = y.abs().amax(-1, keepdim=True) / 127.0
    q = _away(y * torch.where(d != 0, 1.0 / d, torch.zeros_like(d)))
    return {"sum": x, "y": (q * d.half().float()).flatten(-2).half()}


def _rotate(x, cos, sin, halves):
    """x [tokens][heads][dim], cos and sin [tokens][rot / 2]: the first rot dimensions of each head turned."""
    rot = 2 * cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if halves:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((y, x[..., rot:]), -1)


def _q4(x):
    """The values that x's Q4_0 blocks stand for, in fp16: the value furthest from zero (the first of them) is -8."""
    b = x.unflatten(-1, (-1, QK))
    mag = b.abs()
    at = torch.where(mag == mag.amax(-1, keepdim=True), torch.arange(QK, device=x.device), QK).amin(-1, keepdim=True)
    d = torch.gather(b, -1, at) / -8.0
    q = torch.trunc(b * torch.where(d != 0, 1.0 / d, torch.zeros_like(d)) + 8.5).clamp(max=15.0) - 8.0
    return (q * d.half().float()).flatten(-2).half()


def _append(s):
    c, qkv = s["case"], s["qkv"]
    hq, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    q, k, v = qkv.unflatten(-1, (-1, dim)).split((hq, hk, hk), 1)
    cos, sin = s["rope"][s["pos"].long()].chunk(2, 1)
    return {"q": _rotate(q, cos, sin, c["halves"]), "k": _q4(_rotate(k, cos, sin, c["halves"])), "v": _q4(v)}


def _attn(s):
    c = s["case"]
    hq, hk, dim, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    group, n_seq, most = hq // hk, c["seqs"], s["max_new"]
    tiles = s["pages"].view(-1, hk, page // SLAB, 18 * dim)[s["table"].long()]  # [seq][page][head][slab][bytes]
    k, v = (t.permute(0, 2, 1, 3, 4, 5).flatten(2, 4) for t in tile_values(tiles, dim))  # [seq][head][token][dim]
    first, lens = s["q_start"][:-1].long(), s["kv_len"].long()
    new = s["q_start"][1:].long() - first
    i = torch.arange(most, device=k.device)
    rows = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].unflatten(2, (hk, group)).permute(0, 2, 1, 3, 4)  # [seq][head][new][group][dim]
    score = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (most, group)) / math.sqrt(dim)
    end = lens[:, None] - (new[:, None] - 1 - i)  # tokens that the i-th new one may see: those before `end`
    t = torch.arange(k.shape[2], device=k.device)
    see = t < end[..., None]
    if c["window"]:
        see &= t >= end[..., None] - c["window"]
    score = torch.where(see[:, None, :, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (most, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return out[i < new[:, None]]


# ------------------------------------------------------------------ what cannot be done without
def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (4 + 4 + 4 + 34 / 32 + 2) + 4 * case["cols"], "flops": 8 * n}
    hq, hk, dim, n = case["heads"], case["kv_heads"], case["dim"], case["tokens"]
    if case["op"] == "append":
        rows = case["seqs"] * n
        # fp32 rows in, fp32 q out, 18 bytes for 32 values of k and v, and the values these stand for in fp16
        return {"bytes": rows * dim * (4 * (2 * hq + 2 * hk) + 2 * hk * (18 / 32 + 2)) + rows * 4 * (case["rot"] + 2),
                "flops": rows * (3 * (hq + hk) * case["rot"] + 4 * 2 * hk * dim)}
    held = seen = new = 0
    for t in lengths(case):
        m = min(n, t) if t else 1
        new += m
        ends = [max(0, t - (m - 1 - i)) for i in range(m)]
        seen += sum(min(e, case["window"] or e) for e in ends)
        held += ends[-1] - (max(0, ends[0] - case["window"]) if case["window"] else 0)
    return {"bytes": held * hk * dim * 2 * 18 / 32 + new * hq * dim * 8, "flops": 4 * seen * hq * dim}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attn}[case["op"]](case, s)


def _host(t):
    return t.cpu().numpy().astype(np.float64)


def _exact_norm(case, s):
    total = _host(s["x"]) + _host(s["r"])
    y = total * (_host(s["w"]) / np.sqrt(np.square(total).sum(1, keepdims=True) / case["cols"] + EPS))
    blocks = y.reshape(-1, QK)
    step = np.abs(blocks).max(1, keepdims=True) / 127
    code = blocks / np.where(step > 0, step, 1)
    code = np.copysign(np.floor(np.abs(code) + 0.5), code)
    return {"sum": total, "y": (code * step.astype(np.float16).astype(np.float64)).reshape(y.shape)}


def _exact_append(case, s):
    hq, hk, dim, half = case["heads"], case["kv_heads"], case["dim"], case["rot"] // 2
    x = _host(s["qkv"]).reshape(-1, hq + 2 * hk, dim)
    turn = _host(s["rope"])[s["pos"].cpu().numpy()]
    turn = (turn[:, :half] + 1j * turn[:, half:])[:, None]
    a, b = (slice(0, half), slice(half, 2 * half)) if case["halves"] else (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    qk = x[:, :hq + hk]
    z = (qk[..., a] + 1j * qk[..., b]) * turn
    qk[..., a], qk[..., b] = z.real, z.imag
    blocks = x[:, hq:].reshape(-1, QK)
    at = np.argmax(np.abs(blocks), 1)
    step = blocks[np.arange(len(blocks)), at][:, None] / -8
    code = np.minimum(np.floor(blocks / np.where(step != 0, step, 1) + 8.5), 15) - 8
    kv = (code * step.astype(np.float16).astype(np.float64)).reshape(-1, 2, hk, dim)
    return {"q": x[:, :hq], "k": kv[:, 0], "v": kv[:, 1]}


def _exact_attn(case, s):
    hq, hk, dim, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if work(case)["flops"] > 4e11:
        return None
    out, row = [], 0
    pages = s["pages"].view(-1, hk, page // SLAB, 18 * dim)
    where_k, where_v = code_index(dim, "cuda")
    where_d = scale_index(dim, "cuda").repeat_interleave(QK, 1)
    for i, t in enumerate(lengths(case)):
        m = s["new"][i]
        q = s["q"][row:row + m].double()
        row += m
        if t == 0:
            out.append(torch.zeros_like(q))
            continue
        held = pages[s["table"][i, :-(-t // page)].long()]
        got = torch.zeros(m, hq, dim, dtype=torch.float64, device="cuda")
        at = torch.arange(t, device="cuda")
        for h in range(hk):
            tiles = held[:, h].reshape(-1, 18 * dim)
            d = tiles[:, 16 * dim:].contiguous().view(torch.float16).double()
            kv = []
            for n, base, scales in ((where_k, 0, d[:, :dim // 2]), (where_v, 8 * dim, d[:, dim // 2:])):
                byte = tiles[:, (base + n // 2).flatten()].to(torch.int32)
                code = torch.where((n % 2 == 0).flatten(), byte % 16, byte // 16) - 8
                kv.append((code * scales[:, where_d.flatten()]).reshape(-1, dim)[:t])
            for j in range(m):
                end = t - (m - 1 - j)
                low = max(0, end - case["window"]) if case["window"] else 0
                heads = slice(h * (hq // hk), (h + 1) * (hq // hk))
                score = q[j, heads] @ kv[0][low:end].T / math.sqrt(dim)
                got[j, heads] = torch.softmax(score, 1) @ kv[1][low:end]
        out.append(got)
    return torch.cat(out)
