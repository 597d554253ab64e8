"""The operators of drafted trees and bounded memory from their formulas, on the CPU in 64 bits."""
import math

import numpy as np


def tree(rng, m, deep=0.5):
    """Ancestors and itself of each of m drafted tokens, bool [m][m]."""
    sees = np.zeros((m, m), bool)
    for i in range(m):
        parent = i - 1 if rng.random() < deep else int(rng.integers(-1, i)) if i else -1
        if parent >= 0:
            sees[i] = sees[parent]
        sees[i, i] = True
    return sees


def mask_words(sees, words):
    """bool [rows][m] as int32 [rows][words]."""
    bits = np.zeros((len(sees), 32 * words), np.uint64)
    bits[:, :sees.shape[1]] = sees
    return (bits.reshape(len(sees), words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


def tree_visible(n, sees, window):
    """bool [m][n]: which of n keys each row of a tree sees."""
    m = len(sees)
    j = np.arange(n)
    out = np.zeros((m, n), bool)
    for i in range(m):
        p = n - m + max(int(sees[i].sum()) - 1, 0)
        out[i] = (j < n - m) & ((j > p - window) if window else True)
        for c in np.nonzero(sees[i])[0]:
            if 0 <= n - m + c < n:
                out[i, n - m + c] = True
    return out


def causal_visible(n, m, window):
    j, p = np.arange(n), n - m + np.arange(m)[:, None]
    return (j <= p) & ((j > p - window) if window else True)


def attention(q, k, v, scale, visible):
    """q [m][heads][d], k and v [n][kv heads][d], visible [m][n] -> out, lse, sum p |v|, the largest sum
    |q k| of a row."""
    m, heads, d = q.shape
    g = heads // k.shape[1]
    out, size = np.zeros((m, heads, d)), np.zeros((m, heads, d))
    lse, span = np.full((m, heads), -math.inf), np.zeros((m, heads))
    for i in range(m):
        see = np.nonzero(visible[i])[0]
        for h in range(heads if len(see) else 0):
            kk, vv = k[see, h // g], v[see, h // g]
            x = kk @ q[i, h] * scale
            p = np.exp(x - x.max())
            out[i, h], size[i, h] = p @ vv / p.sum(), p @ np.abs(vv) / p.sum()
            lse[i, h] = x.max() + math.log(p.sum())
            span[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * scale
    return out, lse, size, span


def key_weights(w, q, lse, k, scale, window):
    """w [kv heads][n] and rows q [m][heads][d] -> the weights after the call, and what each key's sum may be
    off by in units of a probability's relative error: sum p (1 + |q| |k| + |lse|)."""
    m, heads, _ = q.shape
    n, kvh = k.shape[:2]
    g = heads // kvh
    visible = causal_visible(n, m, window)
    new, size = w.copy(), np.zeros(w.shape)
    new[:, max(0, n - m):] = 0
    for i in range(m):
        for h in range(heads):
            if np.isneginf(lse[i, h]):
                continue
            x = k[:, h // g] @ q[i, h] * scale
            p = np.where(visible[i], np.exp(x - lse[i, h]), 0)
            new[h // g] += p
            size[h // g] += p * (1 + np.abs(k[:, h // g]) @ np.abs(q[i, h]) * scale + abs(lse[i, h]))
    return new, size


def entry(cache, table, page, j, d):
    """Views of key j's four parts in every head: [heads][bytes] each."""
    blk = cache[table[j // page], :, (j % page) // 16]
    r = j % 16
    return [blk[:, a + r * s:a + (r + 1) * s] for a, s in
            ((0, d // 2), (8 * d, d // 2), (16 * d, d // 16), (17 * d, d // 16))]


def move(cache, table, page, d, of, to, heads=slice(None)):
    """Keys `of` to the places `to` in some heads; all are read before any is written."""
    held = [[x[heads].copy() for x in entry(cache, table, page, j, d)] for j in of]
    for j, parts in zip(to, held):
        for x, new in zip(entry(cache, table, page, j, d), parts):
            x[heads] = new


def evict(w, pos, n, last, budget, sink, recent):
    """One head: weights and positions afterwards, and the moves (of, to)."""
    w, pos = w.copy(), pos.copy()
    for j in range(n):
        if pos[j] < 0:
            pos[j] = last - (n - 1 - j)
    if n <= budget:
        return w, pos, [], []

    def better(j):  # the best first
        if pos[j] < sink or pos[j] > last - recent:
            return (0, 0.0, j)
        return (2, 0.0, j) if np.isnan(w[j]) else (1, -float(w[j]), j)

    kept = set(sorted(range(n), key=better)[:budget])
    to = [j for j in range(budget) if j not in kept]
    of = [j for j in range(budget, n) if j in kept]
    w[to], pos[to] = w[of], pos[of]
    pos[budget:n] = -1
    return w, pos, of, to
