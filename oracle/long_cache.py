"""Plain 64-bit forms of the operators for long caches (TEST INFRASTRUCTURE ONLY,
numpy): bounds of cache blocks, the choice of blocks, attention over some blocks,
attention weights per cached token, eviction.

Written from the definitions, one loop per thing the definition names; shares
no code with the CUDA path or the C oracle.
"""
from __future__ import annotations

import math

import numpy as np

BAD_BLOCK, BAD_SEQ_LEN = 1, 2


def _blocks(n, block_size):
    return -(-int(n) // block_size)


def block_bounds(k_cache, table, first_lens, seq_lens, bounds):
    """k_cache [nb, bs, h_kv, d] float64; returns the updated bounds [nb, 2, h_kv, d]."""
    bounds = np.array(bounds, np.float64)
    bs = k_cache.shape[1]
    for b, n in enumerate(int(n) for n in seq_lens):
        first = 0 if first_lens is None else int(first_lens[b])
        if n == 0:
            continue
        for t in range(min(first, n - 1) // bs, _blocks(n, bs)):
            i = int(table[b][t])
            keys = k_cache[i, : min(bs, n - t * bs)]
            bounds[i, 0], bounds[i, 1] = keys.min(0), keys.max(0)  # (numpy's keep NaN)
    return bounds


def block_score(q, low, high):
    """max over the rows of q of sum_d max(q_d low_d, q_d high_d); NaN is +inf."""
    best = -math.inf
    for row in q:
        with np.errstate(invalid="ignore", over="ignore"):
            x = np.maximum(row * low, row * high)
        s = math.fsum(x) if np.isfinite(x).all() else float(x.sum())
        best = max(best, math.inf if math.isnan(s) else s)
    return best


def select_blocks(q, bounds, table, seq_lens, *, block_size, count, first, last):
    """q [B, h_q, d], bounds [nb, 2, h_kv, d] float64: int32 [B, h_kv, count]."""
    B, h_q, _ = q.shape
    h_kv = bounds.shape[2]
    g = h_q // h_kv
    out = np.full((B, h_kv, count), -1, np.int32)
    for b in range(B):
        n = _blocks(seq_lens[b], block_size)
        for j in range(h_kv):
            if n <= count:
                out[b, j, :n] = np.arange(n)
                continue
            some = [t for t in range(n) if t < first or t >= n - last]
            rest = [t for t in range(n) if t not in some]
            score = {t: block_score(q[b, j * g:(j + 1) * g], bounds[table[b][t], 0, j],
                                    bounds[table[b][t], 1, j]) for t in rest}
            rest.sort(key=lambda t: (-score[t], t))
            out[b, j] = sorted(some + rest[: count - len(some)])
    return out


def attend(q, k_cache, v_cache, table, seq_lens, *, scale, selected=None):
    """One query per sequence over all of its tokens, or those of the blocks that
    selected [B, h_kv, count] lists; arrays float64.

    Returns (out, spread, tiny, reach, weights): the first four as step.attend's
    (per row and head), weights[b] [h_q, n] the softmax weights by position.
    """
    B, h_q, d = q.shape
    bs, h_kv = k_cache.shape[1:3]
    g = h_q // h_kv
    out, spread, tiny = (np.zeros(q.shape) for _ in range(3))
    reach = np.zeros((B, h_q))
    weights = []
    for b in range(B):
        n = int(seq_lens[b])
        w = np.zeros((h_q, n))
        for j in range(h_kv):
            t = np.arange(n)
            if selected is not None:
                t = t[np.isin(t // bs, [s for s in selected[b][j] if s >= 0])]
            if not len(t):
                continue
            ids = np.asarray(table[b])[t // bs]
            k, v = k_cache[ids, t % bs, j], v_cache[ids, t % bs, j]
            for h in range(j * g, (j + 1) * g):
                s = scale * (k @ q[b, h])
                if (s == -np.inf).all():
                    continue
                p = np.exp(s - s.max())
                out[b, h] = p @ v / p.sum()
                spread[b, h] = p @ np.abs(v) / p.sum()
                tiny[b, h] = np.abs(v).sum(0) / p.sum()
                reach[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
                w[h, t] = p / p.sum()
        weights.append(w)
    return out, spread, tiny, reach, weights


def add_weights(old, p, table, seq_lens, weighed_lens, *, decay=1.0):
    """old [nb, h_kv, bs] float64, p: attend's weights; the updated array."""
    w = np.array(old, np.float64)
    h_kv, bs = w.shape[1:]
    for b, n in enumerate(int(n) for n in seq_lens):
        g = p[b].shape[0] // h_kv
        done = n - 1 if weighed_lens is None else int(weighed_lens[b])
        for t in range(n):
            at = int(table[b][t // bs]), slice(None), t % bs
            add = p[b][:, t].reshape(h_kv, g).sum(1)
            w[at] = (decay * w[at] if t < done else 0.0) + add
    return w


def evict(k_cache, v_cache, weights, table, seq_lens, *, keep, recent, limit):
    """Arrays of any type; returns (k_cache, v_cache, weights, new_lens, kept)."""
    k, v, w = np.array(k_cache), np.array(v_cache), np.array(weights)
    h_kv, bs = w.shape[1:]
    B = len(seq_lens)
    new, kept = np.zeros(B, np.int32), np.full((B, h_kv, keep), -1, np.int32)
    for b, n in enumerate(int(n) for n in seq_lens):
        if n <= limit:
            continue
        new[b] = keep - n
        slot = [(int(table[b][t // bs]), t % bs) for t in range(n)]
        for j in range(h_kv):
            def rank(t):
                x = float(weights[slot[t][0], j, slot[t][1]])
                return (-math.inf if math.isnan(x) else -x, not math.isnan(x), t)

            old = sorted(range(n - recent), key=rank)[: keep - recent]
            kept[b, j] = sorted(old) + list(range(n - recent, n))
            for r, t in enumerate(kept[b, j]):
                (i, o), (i1, o1) = slot[r], slot[t]
                k[i, o, j], v[i, o, j] = k_cache[i1, o1, j], v_cache[i1, o1, j]
                w[i, j, o] = weights[i1, j, o1]
    return k, v, w, new, kept
