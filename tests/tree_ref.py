"""Plain numpy restatements of the operators on drafted trees and eviction, in 64 bits (the cache's layout and blocks:
tests/block_ref.py)."""
import numpy as np

from tests import block_ref as R


def tree_mask(n, rng, wide=3):
    """[n][n] truth values: token i sees its ancestors and itself; parents anywhere among the `wide` latest or the root."""
    m = np.zeros((n, n), bool)
    for i in range(n):
        if i:
            m[i] = m[max(0, i - 1 - int(rng.integers(0, wide)))]
        m[i, i] = True
    return m


def pack(masks, words):
    """Rows of bits, int32 [rows of all masks][words], of [n][n] truth values a sequence."""
    rows = []
    for m in masks:
        bits = np.zeros((m.shape[0], 32 * words), np.uint64)
        bits[:, :m.shape[1]] = m
        rows.append((bits.reshape(-1, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32))
    return np.concatenate(rows).reshape(-1, words).view(np.int32)


def visible(length, n, i, mask=None, window=0):
    """Truth value of each of the cache's tokens: what new token i of n sees. mask: [n][n] or None (a chain)."""
    t = np.arange(length)
    if mask is None:
        end = length - (n - 1 - i)
        return (t < end) & (t >= (end - window if window else 0))
    base = length - n
    see = t < base
    if window:
        see &= t >= base - max(0, window - int(mask[i].sum()))
    j = t - base
    return see | ((j >= 0) & mask[i][np.clip(j, 0, n - 1)])


def attention(q, q_start, lens, table, k, v, page_tokens, scale, masks=None, window=0):
    """(out, lse, tol_p, tol_v) in 64 bits; the latter two as block_ref.attention's. masks: one a sequence."""
    n_tok, hq, dim = q.shape
    hk = k.shape[1]
    group = hq // hk
    out, lse = np.zeros(q.shape), np.full((n_tok, hq), -np.inf)
    tol_p, tol_v = np.zeros((n_tok, hq)), np.zeros(q.shape)
    for s, length in enumerate(lens):
        n, rows = q_start[s + 1] - q_start[s], slice(q_start[s], q_start[s + 1])
        if n == 0 or length <= 0:
            continue
        see = np.array([visible(length, n, i, None if masks is None else masks[s], window) for i in range(n)])
        some = see.any(1)
        t = np.arange(length)
        page, at = table[s][t // page_tokens], t % page_tokens
        for h in range(hk):
            heads = slice(h * group, (h + 1) * group)
            kk, vv = k[page, h, at], v[page, h, at]
            qq = q[rows, heads].astype(np.float64)
            big_k, big_v = (np.abs(x).reshape(length, -1, R.QK).max(-1) for x in (kk, vv))
            score = np.where(see[:, None], qq @ kk.T * scale, -np.inf)
            top = np.where(some[:, None], score.max(-1, initial=-np.inf), 0)
            e = np.exp(score - top[..., None])
            total = np.where(some[:, None], e.sum(-1), 1)
            lse[rows, heads] = np.where(some[:, None], top + np.log(total), -np.inf)
            p = e / total[..., None]
            # what a row does not see may be no number
            out[rows, heads] = np.array([[pj[see[i]] @ vv[see[i]] for pj in p[i]] for i in range(n)])
            reach = np.abs(qq).reshape(n, group, -1, R.QK).sum(-1) @ big_k.T
            tol_p[rows, heads] = abs(scale) * np.where(see[:, None], reach, 0).max(-1, initial=0)
            tol_v[rows, heads] = np.array([[np.repeat(pj[see[i]] @ big_v[see[i]], R.QK) for pj in p[i]] for i in range(n)])
    return out, lse, tol_p, tol_v


def weights(q, q_start, lens, table, k, page_tokens, scale, lse, masks=None, window=0):
    """(sums, tol): [seq][head][most tokens] of exp(score - lse) over the rows that see a token, in 64 bits, and of each
    |scale| sum |q_e| max|k_block| times it, for the tests' bounds."""
    n_tok, hq, dim = q.shape
    hk = k.shape[1]
    group = hq // hk
    sums = np.zeros((len(lens), hk, max(1, max(lens))))
    tol = np.zeros(sums.shape)
    for s, length in enumerate(lens):
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            row = q_start[s] + i
            t = np.flatnonzero(visible(length, n, i, None if masks is None else masks[s], window))
            if len(t) == 0:
                continue
            page, at = table[s][t // page_tokens], t % page_tokens
            for h in range(hq):
                kk = k[page, h // group, at]
                p = np.exp(kk @ q[row, h].astype(np.float64) * scale - lse[row, h])
                sums[s, h // group, t] += p
                big_k = np.abs(kk).reshape(len(t), -1, R.QK).max(-1)
                reach = abs(scale) * (big_k @ np.abs(q[row, h].astype(np.float64)).reshape(-1, R.QK).sum(-1))
                tol[s, h // group, t] += p * (reach + abs(lse[row, h]) + 16)
    return sums, tol


def evict_index(sums, lens, budget, sinks, recent):
    """int32 [seq][head][budget]: the kept tokens, rising; -1 behind them."""
    n_seq, heads = sums.shape[:2]
    index = np.full((n_seq, heads, budget), -1, np.int32)
    for s, n in enumerate(lens):
        for h in range(heads):
            if n <= budget:
                index[s, h, :max(n, 0)] = np.arange(max(n, 0))
                continue
            rank = np.where(np.isnan(sums[s, h, :n]), -np.inf, sums[s, h, :n].astype(np.float64))
            middle = list(range(sinks, n - recent))
            best = sorted(middle, key=lambda t: (-rank[t], t))[:budget - sinks - recent]
            index[s, h] = sorted(list(range(sinks)) + best + list(range(n - recent, n)))
    return index
