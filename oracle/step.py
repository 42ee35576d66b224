"""Plain 64-bit forms of a serving step's operators (TEST INFRASTRUCTURE ONLY,
numpy): the paged plan, rotary positions, and attention of packed rows over a
paged cache with a window and kept first tokens.

Written from the definitions, one loop per thing the definition names; shares
no code with the CUDA path or the C oracle.
"""
from __future__ import annotations

import numpy as np

BAD_BLOCK, BAD_SEQ_LEN, NO_ROOM = 1, 2, 8


def paged_plan(cached, new, table, free, count, *, block_size, max_tokens):
    """Returns a dict of the updated arrays and the error flag."""
    cached, new = [int(c) for c in cached], [int(n) for n in new]
    table, free = np.array(table), np.array(free)
    B, M = table.shape
    nb, room, flag = len(free), M * block_size, 0
    seq, move = [], []
    for c, n in zip(cached, new):
        if not 0 <= c <= room or not 0 <= c + n <= room:
            flag |= BAD_SEQ_LEN
            c, n = (c if 0 <= c <= room else 0), 0
        seq.append(c)
        move.append(n)

    def blocks(n):
        return -(-n // block_size)

    back = [(b, k) for b in range(B) for k in range(blocks(seq[b] + move[b]), blocks(seq[b]))
            if move[b] < 0]
    want = [(b, k) for b in range(B) for k in range(blocks(seq[b]), blocks(seq[b] + move[b]))
            if move[b] > 0]
    rows = [(b, seq[b] + i) for b in range(B) for i in range(max(0, move[b]))]
    slots, positions = np.full(max_tokens, -1, np.int32), np.full(max_tokens, -1, np.int32)
    start = np.zeros(B + 1, np.int32)
    if not 0 <= count <= nb or len(back) > nb - count:
        return dict(table=table, free=free, count=count, seq_lens=np.array(seq, np.int32),
                    q_start=start, slots=slots, positions=positions, flag=flag | BAD_BLOCK)
    grows = len(want) <= count + len(back) and len(rows) <= max_tokens
    if not grows:
        flag |= NO_ROOM
    for b, k in back:
        if not 0 <= table[b, k] < nb:
            flag |= BAD_BLOCK
        free[count] = table[b, k]
        count += 1
    if grows:
        for b, k in want:
            count -= 1
            if not 0 <= free[count] < nb:
                flag |= BAD_BLOCK
            table[b, k] = free[count]
        for i, (b, p) in enumerate(rows):
            positions[i] = p
            if 0 <= table[b, p // block_size] < nb:
                slots[i] = table[b, p // block_size] * block_size + p % block_size
            else:
                flag |= BAD_BLOCK
            start[b + 1] = i + 1
        start = np.maximum.accumulate(start)
    after = [c + (n if n < 0 or grows else 0) for c, n in zip(seq, move)]
    return dict(table=table, free=free, count=count, seq_lens=np.array(after, np.int32),
                q_start=start, slots=slots, positions=positions, flag=flag)


def rope(x, positions, inv_freq, axis, interleaved):
    """x [T, h, d] float64, positions [axes, T]: the rotated heads."""
    y = np.array(x, np.float64)
    r = len(inv_freq)
    for i, (f, a) in enumerate(zip(inv_freq, axis)):
        j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        angle = np.asarray(positions[a], np.float64) * f
        c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
        y[:, :, j] = x[:, :, j] * c - x[:, :, k] * s
        y[:, :, k] = x[:, :, j] * s + x[:, :, k] * c
    return y


def visible(p, window, sinks):
    """The positions that the row at position p sees."""
    t = np.arange(p + 1)
    return t if not window else t[(t > p - window) | (t < sinks)]


def attend(q, k_cache, v_cache, table, q_start, seq_lens, *, scale, window=0, sinks=0):
    """Attention of packed rows over a paged cache, all arrays float64.

    Returns (out, spread, tiny, reach): the result [T, h_q, d]; per row and
    head, sum p |v| / sum p [T, h_q, d] and sum |v| / sum e^(s - max)
    [T, h_q, d]; and max over the seen tokens of |scale| sum |q| |k| [T, h_q]:
    what a rounding of p, a lost p and an error of a score can move.  Rows
    outside every sequence are NaN.
    """
    T, h_q, d = q.shape
    nb, bs, h_kv, _ = k_cache.shape
    g = h_q // h_kv
    out, spread, tiny = (np.full(q.shape, np.nan) for _ in range(3))
    reach = np.full((T, h_q), np.nan)
    for b, n_all in enumerate(seq_lens):
        a, e = int(q_start[b]), int(q_start[b + 1])
        ids = np.asarray(table[b][: -(-int(n_all) // bs)], np.int64)
        if e == a:
            continue
        used = set()
        for i in range(a, e):
            used.update((visible(int(n_all) - e + i, window, sinks) // bs).tolist())
        K = np.zeros((len(ids) * bs, h_kv, d))
        V = np.zeros((len(ids) * bs, h_kv, d))
        for u in used:  # only blocks that some row sees are looked at
            K[u * bs:(u + 1) * bs], V[u * bs:(u + 1) * bs] = k_cache[ids[u]], v_cache[ids[u]]
        for i in range(a, e):
            t = visible(int(n_all) - e + i, window, sinks)
            for h in range(h_q):
                if not len(t):
                    out[i, h] = spread[i, h] = tiny[i, h] = 0.0
                    reach[i, h] = 0.0
                    continue
                k, v = K[t, h // g], V[t, h // g]
                s = scale * (k @ q[i, h])
                p = np.exp(s - s.max())
                out[i, h] = p @ v / p.sum()
                spread[i, h] = p @ np.abs(v) / p.sum()
                tiny[i, h] = np.abs(v).sum(0) / p.sum()
                reach[i, h] = abs(scale) * (np.abs(k) @ np.abs(q[i, h])).max()
    return out, spread, tiny, reach
