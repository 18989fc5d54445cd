"""Drafted trees and eviction on the paged 4-bit cache, as cases to measure.

Four operators, in their plain form (elementary torch operations in fp32) and through the library:

  tree     attention of a tree of drafted tokens over the cache: every new token sees what was cached before them (or
           the last of it, with a window) and, of the new ones, those that its row of bits names: its ancestors
  accept   the accepted path of a tree moves down to follow what was cached before: the cache holds one line of tokens
           again
  weights  every cached token's attention weight, summed over the query heads of its kv head and over the new tokens,
           added to what earlier steps gave it
  evict    of each kv head the tokens with the largest sums, the first ones and the latest ones go to pages of their
           own, in their order; the others are forgotten

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


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a few drafted tokens early in a sequence's life, a head of its own for every query head: latency alone
        {"name": "tree 1x4 333 d64", "op": "tree", "seqs": 1, "tokens": 4, "heads": 16, "kv_heads": 16, "dim": 64,
         "page": 32, "longest": 333, "shortest": 333, "window": 0},
        # an ordinary tree, wide heads of which eight share a kv head
        {"name": "tree 1x12 2011 d256", "op": "tree", "seqs": 1, "tokens": 12, "heads": 16, "kv_heads": 2, "dim": 256,
         "page": 64, "longest": 2011, "shortest": 2011, "window": 0},
        # a serving batch of ragged lengths and trees, a sliding window
        {"name": "tree 8x25 ragged window", "op": "tree", "seqs": 8, "tokens": 25, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "longest": 8191, "shortest": 3, "window": 4096},
        # a large tree over a long context
        {"name": "tree 1x64 65521", "op": "tree", "seqs": 1, "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "longest": 65521, "shortest": 65521, "window": 0},
        # one sequence's path of five
        {"name": "accept 1 path d256", "op": "accept", "seqs": 1, "tokens": 12, "heads": 16, "kv_heads": 2, "dim": 256,
         "page": 64, "longest": 2011, "shortest": 2011},
        # a serving batch's paths
        {"name": "accept 48 paths", "op": "accept", "seqs": 48, "tokens": 64, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "longest": 4096, "shortest": 70},
        # one decode token early in a sequence's life
        {"name": "weights 1x777 d256", "op": "weights", "seqs": 1, "tokens": 1, "heads": 16, "kv_heads": 2, "dim": 256,
         "page": 64, "longest": 777, "shortest": 777, "window": 0},
        # one token of a very long context
        {"name": "weights 1x130975", "op": "weights", "seqs": 1, "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "longest": 130975, "shortest": 130975, "window": 0},
        # a serving batch's decode step
        {"name": "weights 48 ragged 16384", "op": "weights", "seqs": 48, "tokens": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "longest": 16384, "shortest": 0, "window": 0},
        # the weights that a prompt's last chunk gives what came before it
        {"name": "weights chunk 256x8192", "op": "weights", "seqs": 1, "tokens": 256, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "longest": 8192, "shortest": 8192, "window": 0},
        # a small cache back to its budget
        {"name": "evict 1x1500 to 1000 d64", "op": "evict", "seqs": 1, "heads": 8, "kv_heads": 4, "dim": 64, "page": 32,
         "longest": 1500, "shortest": 1500, "budget": 1000, "sinks": 4, "recent": 200},
        # long contexts of a batch, one of them short enough to stay as it is
        {"name": "evict 4 ragged 65536 to 16000", "op": "evict", "seqs": 4, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 64, "longest": 65536, "shortest": 9000, "budget": 16000, "sinks": 16, "recent": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "weights", "evict", "accept"])
    dim = rng.choice([64, 96, 128, 128, 192, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": rng.choice([16, 32, 64, 128])}
    if op == "accept":
        seqs = _log(rng, 1, 48)
        return {**case, "seqs": seqs, "tokens": _log(rng, 2, 64), "longest": _log(rng, 80, 4096), "shortest": 70}
    if op == "evict":
        seqs = _log(rng, 1, 16)
        longest = _log(rng, 40, max(41, min(65536, (1 << 28) // (seqs * kv_heads * dim))))
        budget = max(8, int(longest * rng.uniform(0.1, 0.9)))
        return {**case, "seqs": seqs, "longest": longest, "shortest": longest if seqs == 1 else longest // rng.choice([2, 8]),
                "budget": budget, "sinks": rng.choice([0, 1, 4]), "recent": rng.choice([0, budget // 8, budget // 2])}
    kind = rng.choice(["one", "few", "many"]) if op == "weights" else rng.choice(["few", "few", "many"])
    seqs, tokens = {"one": (_log(rng, 1, 48), 1), "few": (_log(rng, 1, 16), rng.randint(2, 16)),
                    "many": (rng.randint(1, 2), _log(rng, 17, 64))}[kind]
    # a drawn case costs at most a quarter or so of the largest listed one
    most = {"one": 8 * 128 * (1 << 19), "few": 8 * 128 * (1 << 15), "many": 8 * 128 * (1 << 13)}[kind]
    longest = max(tokens + 1, _log(rng, 20, max(21, min(131072, 4 * most // (seqs * heads * dim)))))
    return {**case, "seqs": seqs, "tokens": tokens, "longest": longest,
            "shortest": longest if seqs == 1 else longest // rng.choice([2, 8, 50]),
            "window": rng.choice([0, 0, 0, max(1, longest // 3)])}


def lengths(case):
    """Tokens of each sequence in the cache, the new ones among them: log-spread, the longest and the shortest there."""
    n, lo, hi = case["seqs"], case["shortest"], case["longest"]
    if n == 1:
        return [hi]
    rng = random.Random(1009 * n + hi)
    mid = [min(hi, max(lo, _log(rng, max(lo, hi // 16, 1), max(hi, 2)))) for _ in range(n - 2)]
    return [hi] + mid + [lo]


def new_tokens(case):
    """New tokens of each sequence: the first has as many as the call allows, of trees the others may have fewer."""
    lens, n = lengths(case), case["tokens"]
    rng = random.Random(31 * n + lens[0])
    return [min(n if i == 0 or case["op"] == "weights" else rng.randint(1, n), t) if t else (1 if n == 1 else 0)
            for i, t in enumerate(lens)]


def parents(n, rng):
    """A tree of n drafted tokens in the order of their depths: token 0 is the root (the last token that was sampled),
    every other's parent comes before it. Levels grow to about a quarter of the tree."""
    out, level = [-1], [0]
    while len(out) < n:
        want = min(n - len(out), max(1, min(n // 4, 2 * len(level) + rng.randint(0, 2))))
        of = sorted(rng.choice(level) for _ in range(want))
        level = list(range(len(out), len(out) + want))
        out += of
    return out


def ancestors(tree):
    """[n][n] truth values: token i sees token j, itself among them."""
    m = np.zeros((len(tree), len(tree)), dtype=bool)
    for i, p in enumerate(tree):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def words(mask, n_words):
    """[n][n] truth values as [n][n_words] words of 32 bits, the lowest first."""
    bits = np.zeros((mask.shape[0], 32 * n_words), dtype=np.uint64)
    bits[:, :mask.shape[1]] = mask
    w = (bits.reshape(mask.shape[0], n_words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def path_of(n, rng):
    """An accepted path of a drafted tree: the root, then one token a level. Its tokens but the first lie behind the
    place that the path moves to, as in a tree that is wider than deep."""
    steps = rng.randint(1, max(1, min(8, n // 2)))
    rest = sorted(rng.sample(range(steps, n), steps - 1)) if steps > 1 else []
    return [0] + rest


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


def token_parts(tiles, dim):
    """Tiles of bytes [..., 18 dim] token by token: K's and V's codes [..., SLAB, dim] and scales [..., SLAB, dim / QK],
    the scales as the 16-bit numbers that they are stored as."""
    scales = tiles[..., 16 * dim:].contiguous().view(torch.int16)
    at = scale_index(dim, tiles.device)
    codes, steps = [], []
    for which, n in enumerate(code_index(dim, tiles.device)):
        c = tiles[..., 8 * dim * which:8 * dim * (which + 1)]
        codes.append(torch.stack((c & 15, c >> 4), -1).flatten(-2)[..., n])
        steps.append(scales[..., which * dim // 2:(which + 1) * dim // 2][..., at])
    return codes, steps


def tiles_of(codes, steps, dim):
    """The tiles [..., 18 dim] of such parts."""
    lead, device = codes[0].shape[:-2], codes[0].device
    out = torch.empty(*lead, 18 * dim, dtype=torch.uint8, device=device)
    at = scale_index(dim, device).flatten()
    for which, n in enumerate(code_index(dim, device)):
        nib = torch.empty(*lead, SLAB * dim, dtype=torch.uint8, device=device)
        nib[..., n.flatten()] = codes[which].flatten(-2)
        out[..., 8 * dim * which:8 * dim * (which + 1)] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        half = torch.empty(*lead, SLAB * dim // QK, dtype=torch.int16, device=device)
        half[..., at] = steps[which].flatten(-2)
        out[..., (16 + which) * dim:(17 + which) * dim] = half.view(torch.uint8)
    return out


def tile_values(tiles, dim, which):
    """fp32 K (which 0) or V (1), [..., SLAB, dim], of tiles of bytes [..., 18 dim]."""
    d = tiles[..., 16 * dim:].contiguous().view(torch.float16)[..., which * dim // 2:(which + 1) * dim // 2]
    d = d[..., scale_index(dim, tiles.device)].float()
    codes = tiles[..., 8 * dim * which:8 * dim * (which + 1)]
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)[..., code_index(dim, tiles.device)[which]]
    return ((nib.float() - 8.0).unflatten(-1, (dim // QK, QK)) * d[..., None]).flatten(-2)


# ------------------------------------------------------------------ inputs
def _cache(s, case, lens, g):
    """Pages in any order for these lengths, of codes and scales at random."""
    hk, dim, page = case["kv_heads"], case["dim"], case["page"]
    held = [max(1, -(-t // page)) for t in lens]
    order = torch.randperm(sum(held), generator=g, device="cuda").to(torch.int32).tolist()
    table = np.zeros((len(lens), max(held)), dtype=np.int32)
    for i, h in enumerate(held):
        table[i, :h] = [order.pop() for _ in range(h)]
    s["table"] = torch.from_numpy(table).cuda()
    s["pages"] = torch.randint(0, 256, (sum(held) * hk * page // SLAB * 18 * dim,), generator=g, device="cuda", dtype=torch.uint8)
    tiles = s["pages"].view(-1, 18 * dim)
    d = torch.rand(tiles.shape[0], dim, generator=g, device="cuda") * 0.2 + 0.1
    d = torch.where(torch.rand(d.shape, generator=g, device="cuda") < 0.5, -d, d).half()
    tiles[:, 16 * dim:] = d.view(torch.uint8)
    s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    lens, hq, hk, dim = lengths(case), case["heads"], case["kv_heads"], case["dim"]
    s = {"case": case, "max_len": max(lens)}
    _cache(s, case, lens, g)
    if case["op"] in ("tree", "weights"):
        new = new_tokens(case)
        s["q"] = 2.0 * torch.randn(sum(new), hq, dim, generator=g, device="cuda")
        s["q_start"] = torch.tensor(np.concatenate(([0], np.cumsum(new))), dtype=torch.int32, device="cuda")
        s["max_new"] = max(new)
    if case["op"] == "tree":
        rng, n_words = random.Random(seed), -(-max(new) // 32)
        s["seen"] = torch.from_numpy(np.concatenate([words(ancestors(parents(n, rng)), n_words) for n in new if n])).cuda()
    if case["op"] == "weights":
        # what the attention of the same step wrote, and the sums of the steps before it
        s["lse"] = _attention_scores(s)[1]
        s["sums"] = torch.exp(2.0 * torch.randn(len(lens), hk, max(lens), generator=g, device="cuda") - 4.0)
    if case["op"] == "accept":
        new, rng = new_tokens(case), random.Random(seed)
        paths = [path_of(n, rng) for n in new]
        s["base"] = torch.tensor([t - n for t, n in zip(lens, new)], dtype=torch.int32, device="cuda")
        path = np.full((len(lens), case["tokens"]), -1, dtype=np.int32)
        for i, p in enumerate(paths):
            path[i, :len(p)] = p
        s["path"] = torch.from_numpy(path).cuda()
        s["n_path"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    if case["op"] == "evict":
        # weights that add up over a context: few large ones, many that never counted
        sums = torch.exp(3.0 * torch.randn(len(lens), hk, max(lens), generator=g, device="cuda"))
        s["sums"] = torch.where(torch.rand(sums.shape, generator=g, device="cuda") < 0.2, torch.zeros_like(sums), sums)
        held = [-(-min(t, case["budget"]) // case["page"]) for t in lens]
        table = np.zeros((len(lens), max(held)), dtype=np.int32)
        order = torch.randperm(sum(held), generator=g, device="cuda").to(torch.int32).tolist()
        for i, h in enumerate(held):
            table[i, :h] = [order.pop() for _ in range(h)]
        s["to_table"] = torch.from_numpy(table).cuda()
        s["to_pages"] = torch.zeros(sum(held) * hk * case["page"] // SLAB * 18 * dim, dtype=torch.uint8, device="cuda")
    if own:
        _own_prepare(s)
    return s


def _own_prepare(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    c = s["case"]
    hq, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    s["cache"] = Z.KVCache(s["pages"], c["page"], hk, dim, s["table"])
    if c["op"] == "tree":
        s["out"] = torch.empty(s["q"].shape, device="cuda")
        s["lse"] = torch.empty(s["q"].shape[:2], device="cuda")
        s["workspace"] = Z.attn_q4_0_workspace(s["cache"], hq, s["max_new"], s["max_len"])
    if c["op"] == "weights":
        s["sums_out"] = torch.zeros_like(s["sums"])
    if c["op"] == "accept":
        s["len_out"] = torch.empty_like(s["base"])
    if c["op"] == "evict":
        s["to"] = Z.KVCache(s["to_pages"], c["page"], hk, dim, s["to_table"])
        shape = (c["seqs"], hk, c["budget"])
        s["index"], s["sums_out"] = torch.empty(shape, dtype=torch.int32, device="cuda"), torch.empty(shape, device="cuda")
        s["len_out"] = torch.empty_like(s["kv_len"])


# ------------------------------------------------------------------ the operators
def run(s):
    op = s["case"]["op"]
    if own:
        return {"tree": _own_tree, "accept": _own_accept, "weights": _own_weights, "evict": _own_evict}[op](s)
    return {"tree": _tree, "accept": _accept, "weights": _weights, "evict": _evict}[op](s)


def _own_tree(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    Z.attn_tree_q4_0(s["cache"], s["q"], s["q_start"], s["kv_len"], s["max_new"], s["max_len"], seen=s["seen"],
                     window=s["case"]["window"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_accept(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    Z.kv_accept_q4_0(s["cache"], s["base"], s["path"], s["n_path"], len_out=s["len_out"])
    return {"len": s["len_out"], "pages": s["pages"]}


def _own_weights(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    Z.attn_weights_q4_0(s["cache"], s["q"], s["q_start"], s["kv_len"], s["lse"], s["max_new"], s["max_len"],
                        window=s["case"]["window"], sums=s["sums"], out=s["sums_out"])
    return {"sums": s["sums_out"]}


def _own_evict(s):
    from gguf_block_quant_gb300 import zdmmv as Z
    c = s["case"]
    Z.kv_evict_q4_0(s["cache"], s["to"], s["kv_len"], s["sums"], c["budget"], s["max_len"], sinks=c["sinks"],
                    recent=c["recent"], index=s["index"], sums_out=s["sums_out"], len_out=s["len_out"])
    return {"index": s["index"], "sums": s["sums_out"], "len": s["len_out"], "pages": s["to_pages"]}


def _sequences(s, which):
    """fp32 K (which 0) or V (1) of all sequences, [seq][head][token][dim], as far as the page table goes."""
    c = s["case"]
    tiles = s["pages"].view(-1, c["kv_heads"], c["page"] // SLAB, 18 * c["dim"])[s["table"].long()]
    return tile_values(tiles, c["dim"], which).permute(0, 2, 1, 3, 4, 5).flatten(2, 4)


def _attention_scores(s):
    """Scores [seq][head][new token, query head of the group][token], -inf where nothing is seen, and the logarithm of
    the sum of their exponentials, [row][query head]."""
    c = s["case"]
    hq, hk, dim, most = c["heads"], c["kv_heads"], c["dim"], s["max_new"]
    k = _sequences(s, 0)
    first, lens = s["q_start"][:-1].long(), s["kv_len"].long()
    new = s["q_start"][1:].long() - first
    i = torch.arange(most, device=k.device)
    rows = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].unflatten(2, (hk, hq // hk)).permute(0, 2, 1, 3, 4)  # [seq][head][new][group][dim]
    score = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (most, hq // hk)) / math.sqrt(dim)
    t = torch.arange(k.shape[2], device=k.device)
    base = (lens - new)[:, None, None]
    if "seen" in s:
        bits = s["seen"][rows].long() & 0xFFFFFFFF                        # [seq][new][words]
        j = (t - base).clamp(min=0)                                       # [seq][1][token]: which of the new ones it is
        word = torch.gather(bits, 2, (j // 32).clamp(max=bits.shape[2] - 1).expand(-1, most, -1))
        mine = (word >> (j % 32)) & 1
        see = torch.where(t < base, torch.ones_like(mine), mine) == 1
        see &= t < lens[:, None, None]
        if c["window"]:
            ahead = torch.where((t >= base) & (t < lens[:, None, None]), mine, torch.zeros_like(mine)).sum(-1, keepdim=True)
            see &= (t >= base) | (t >= base - (c["window"] - ahead).clamp(min=0))
    else:
        end = (lens[:, None] - (new[:, None] - 1 - i))[..., None]
        see = t < end
        if c["window"]:
            see &= t >= end - c["window"]
    score = torch.where(see[:, None, :, None], score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    lse = (top + torch.log(torch.exp(score - top).sum(-1, keepdim=True)))[..., 0]
    live = i < new[:, None]
    lse = lse.permute(0, 2, 1, 3).flatten(2, 3)[live]
    return score, lse, live


def _tree(s):
    c = s["case"]
    score, lse, live = _attention_scores(s)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    out = torch.matmul(p.flatten(2, 3), _sequences(s, 1)).unflatten(2, (s["max_new"], c["heads"] // c["kv_heads"]))
    return {"out": out.permute(0, 2, 1, 3, 4).flatten(2, 3)[live], "lse": lse}


def _weights(s):
    score, _, live = _attention_scores(s)
    n_seq, hk, most, group = score.shape[:4]
    lse = torch.zeros(n_seq, most, hk * group, device=score.device)
    lse[live] = s["lse"]
    p = torch.exp(score - lse.unflatten(2, (hk, group)).permute(0, 2, 1, 3)[..., None])
    p = torch.where(live[:, None, :, None, None] & (score > -math.inf), p, torch.zeros_like(p))
    add = p.sum((2, 3))[..., :s["sums"].shape[2]]
    t = torch.arange(add.shape[2], device=add.device)
    lens = s["kv_len"].long()
    base = lens - (s["q_start"][1:] - s["q_start"][:-1]).long()
    before = torch.where(t < base[:, None, None], s["sums"], torch.zeros_like(s["sums"]))
    return {"sums": torch.where(t < lens[:, None, None], before + add, torch.zeros_like(add))}


def _accept(s):
    c = s["case"]
    hk, dim, page = c["kv_heads"], c["dim"], c["page"]
    pages = s["pages"].view(-1, hk, page // SLAB, 18 * dim)
    j = torch.arange(c["tokens"], device="cuda")
    seq, j = ((j < s["n_path"][:, None]) & (s["path"] != j)).nonzero(as_tuple=True)
    frm, to = s["base"][seq] + s["path"][seq, j], s["base"][seq] + j
    at = [(s["table"][seq, (t // page).long()].long(), (t % page // SLAB).long(), (t % SLAB).long()) for t in (frm, to)]
    (p0, u0, r0), (p1, u1, r1) = at
    codes, steps = token_parts(pages[p0, :, u0], dim)                      # [move][head][SLAB][...]
    take = torch.arange(len(seq), device="cuda")
    # bytes hold two values of one token, so a token's bytes can be put by themselves
    index = code_index(dim, "cuda")
    for which in (0, 1):
        c4 = codes[which][take, :, r0]                                     # [move][head][dim]
        n = index[which][r1]                                               # [move][dim]
        where = 8 * dim * which + n[:, 0::2] // 2
        pages[p1[:, None, None], torch.arange(hk, device="cuda")[:, None], u1[:, None, None], where[:, None]] = \
            c4[..., 0::2] | (c4[..., 1::2] << 4)
        half = pages.view(torch.int16)
        where = (16 + which) * dim // 2 + scale_index(dim, "cuda")[r1]
        half[p1[:, None, None], torch.arange(hk, device="cuda")[:, None], u1[:, None, None], where[:, None]] = \
            steps[which][take, :, r0]
    return {"len": s["base"] + s["n_path"], "pages": s["pages"]}


def _evict(s):
    c = s["case"]
    hk, dim, page, budget = c["kv_heads"], c["dim"], c["page"], c["budget"]
    lens = s["kv_len"].long()[:, None, None]
    t = torch.arange(s["sums"].shape[2], device="cuda")
    always = (t < c["sinks"]) | (t >= lens - c["recent"])
    rank = torch.where(always, torch.full_like(s["sums"], math.inf), s["sums"])
    rank = torch.where(t < lens, rank, torch.full_like(rank, -math.inf))
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    keep = torch.zeros_like(rank, dtype=torch.bool).scatter_(-1, order, True) & (t < lens)
    kept = lens.clamp(max=budget)
    index = torch.sort(torch.where(keep, t, t.numel()), dim=-1).values[..., :budget]
    if index.shape[-1] < budget:
        index = torch.cat((index, torch.full((*index.shape[:2], budget - index.shape[-1]), t.numel(), device="cuda")), -1)
    live = torch.arange(budget, device="cuda") < kept
    index = torch.where(live, index, torch.full_like(index, -1))
    some = index.clamp(min=0)
    sums = torch.where(live, torch.gather(s["sums"], 2, some), torch.zeros(index.shape, device="cuda"))
    # whole tiles of 16 tokens, zeros behind the last one
    n_tiles = -(-budget // SLAB)
    some = torch.cat((index, index.new_full((*index.shape[:2], n_tiles * SLAB - budget), -1)), -1)
    to_pages = s["to_pages"].view(-1, hk, page // SLAB, 18 * dim)
    pages = s["pages"].view(-1, hk, page // SLAB, 18 * dim)
    for i in range(c["seqs"]):
        codes, steps = token_parts(pages[s["table"][i].long()].permute(1, 0, 2, 3).flatten(1, 2), dim)
        at = some[i].clamp(min=0)[..., None]
        put = [[torch.where(some[i][..., None] >= 0, torch.gather(x.flatten(1, 2), 1, at.expand(-1, -1, x.shape[-1])), 0)
                .unflatten(1, (n_tiles, SLAB)) for x in xs] for xs in (codes, steps)]
        tiles = tiles_of(*put, dim)                                        # [head][tile][bytes]
        k = torch.arange(n_tiles, device="cuda")
        k = k[k * SLAB < kept[i, 0, 0]]
        dst = s["to_table"][i, k * SLAB // page].long()
        to_pages[dst, :, k % (page // SLAB)] = tiles[:, k].transpose(0, 1)
    return {"index": index.int(), "sums": sums, "len": kept[:, 0, 0].int(), "pages": s["to_pages"]}


# ------------------------------------------------------------------ what cannot be done without
def work(case):
    hq, hk, dim, lens = case["heads"], case["kv_heads"], case["dim"], lengths(case)
    token = 2 * dim * 18 / 32  # bytes of a token of a kv head, K and V
    if case["op"] == "accept":
        moved = sum(len(path_of(n, random.Random(i))) - 1 for i, n in enumerate(new_tokens(case)))
        return {"bytes": moved * hk * 2 * token + 12 * len(lens), "flops": 0}
    if case["op"] == "evict":
        kept = sum(min(t, case["budget"]) for t in lens)
        return {"bytes": hk * (4 * sum(lens) + kept * (2 * token + 12)), "flops": 0}
    held = seen = rows = 0
    for t, m in zip(lens, new_tokens(case)):
        rows += m
        w = case["window"]
        if case["op"] == "tree":
            depth = ancestors(parents(m, random.Random(t))).sum(1).tolist() if m else []
            see = [min(t - m, max(0, w - d)) if w else t - m for d in depth]
            seen += sum(a + d for a, d in zip(see, depth))
            held += max(see, default=0) + m
        else:
            ends = [max(0, t - (m - 1 - i)) for i in range(m)]
            seen += sum(min(e, w or e) for e in ends)
            held += ends[-1] - (max(0, ends[0] - w) if w else 0) if m else 0
    if case["op"] == "tree":
        return {"bytes": held * hk * token + rows * hq * (8 * dim + 4) + rows * 4 * -(-case["tokens"] // 32),
                "flops": 4 * seen * hq * dim}
    return {"bytes": held * hk * token / 2 + sum(lens) * hk * 8 + rows * hq * (4 * dim + 4), "flops": 2 * seen * hq * dim}


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"tree": _exact_attention, "weights": _exact_attention, "accept": _exact_accept, "evict": _exact_evict}[case["op"]](case, s)


def _exact_tokens(case, s, i, h, n, which):
    """fp64 K (which 0) or V (1) of the first n tokens of sequence i, kv head h."""
    dim, page, nb = case["dim"], case["page"], case["dim"] // QK
    held = s["pages"].view(-1, case["kv_heads"], page // SLAB, 18 * dim)[s["table"][i, :-(-n // page)].long(), h].reshape(-1, 18 * dim)
    where = code_index(dim, held.device)[which].flatten()
    byte = held[:, 8 * dim * which + where // 2].to(torch.int32)
    code = torch.where(where % 2 == 0, byte % 16, byte // 16) - 8
    d = held[:, (16 + which) * dim:(17 + which) * dim].contiguous().view(torch.float16).double()
    d = d[:, scale_index(dim, held.device).flatten()].reshape(-1, SLAB, nb).repeat_interleave(QK, 2)
    return (code.reshape(-1, SLAB, dim) * d).reshape(-1, dim)[:n]


def _exact_attention(case, s):
    hq, hk, dim = case["heads"], case["kv_heads"], case["dim"]
    if work(case)["flops"] > 4e11:
        return None
    rows, starts, group = s["q"].double(), s["q_start"].tolist(), hq // hk
    out, lse = torch.zeros_like(rows), torch.full(rows.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    sums = None if case["op"] == "tree" else torch.zeros(s["sums"].shape, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lengths(case)):
        a, b = starts[i], starts[i + 1]
        if n == 0:
            continue
        m = b - a
        see = torch.ones(m, n, dtype=torch.bool, device="cuda")
        for j in range(m):
            if case["op"] == "tree":
                bits = [w & 0xFFFFFFFF for w in s["seen"][a + j].tolist()]
                mine = [k for k in range(m) if bits[k // 32] >> (k % 32) & 1]
                see[j, n - m:] = False
                see[j, [n - m + k for k in mine]] = True
                if case["window"]:
                    see[j, :max(0, n - m - max(0, case["window"] - len(mine)))] = False
            else:
                end = n - (m - 1 - j)
                see[j, end:] = False
                if case["window"]:
                    see[j, :max(0, end - case["window"])] = False
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            score = rows[a:b, heads].reshape(-1, dim) @ _exact_tokens(case, s, i, h, n, 0).T / math.sqrt(dim)
            score = score.view(m, group, n).masked_fill(~see[:, None], -math.inf)
            if case["op"] == "tree":
                lse[a:b, heads] = torch.logsumexp(score, -1)
                p = torch.exp(score - lse[a:b, heads, None]).nan_to_num(0.0)
                out[a:b, heads] = p @ _exact_tokens(case, s, i, h, n, 1)
            else:
                p = torch.exp(score - s["lse"][a:b, heads, None].double())
                sums[i, h, :n] = torch.where(see[:, None], p, torch.zeros_like(p)).sum((0, 1))
                sums[i, h, :n - m] += s["sums"][i, h, :n - m].double()
    return {"out": out, "lse": lse} if case["op"] == "tree" else {"sums": sums}


def _exact_accept(case, s):
    return {"len": (s["base"] + s["n_path"]).cpu().numpy(), "pages": None}


def _exact_evict(case, s):
    budget, hk = case["budget"], case["kv_heads"]
    sums = s["sums"].cpu().numpy()
    index = np.full((case["seqs"], hk, budget), -1, dtype=np.int32)
    kept = np.zeros(index.shape)
    lens = lengths(case)
    for i, n in enumerate(lens):
        m = min(n, budget)
        for h in range(hk):
            if n <= budget:
                index[i, h, :m] = np.arange(m)
            else:
                middle = np.arange(case["sinks"], n - case["recent"])
                # the largest sums first, of equal ones the lowest index
                best = middle[np.lexsort((middle, -sums[i, h, middle].astype(np.float64)))][:budget - case["sinks"] - case["recent"]]
                index[i, h] = np.sort(np.concatenate((np.arange(case["sinks"]), best, np.arange(n - case["recent"], n))))
            kept[i, h, :m] = sums[i, h, index[i, h, :m]]
    return {"index": index, "sums": kept, "len": np.minimum(lens, budget).astype(np.int32), "pages": None}
