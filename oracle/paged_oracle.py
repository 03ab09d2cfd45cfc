"""CPU oracle of the paged grouped-query cache: attention with score options, append, eviction.

TEST INFRASTRUCTURE ONLY, like lsa_oracle: plain numpy in float64 (whole numbers for the
tables), written from the definitions in include/lsa.h and sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def seen_positions(block_pos, n, tail, prefix=0, doc_start=0, window=0):
    """(entry, slot, position) of every position that the newest token sees, in order."""
    x_b = PAGE * int(block_pos[n - 1]) + tail - 1
    low = doc_start
    if window > 0:
        low = max(low, x_b - window + 1)
    slots = [(j, t) for j in range(n) for t in range(tail if j == n - 1 else PAGE)]
    at = [(j, t, PAGE * int(block_pos[j]) + t) for j, t in slots]
    return [p for p in at if p[2] < prefix or p[2] >= low], x_b


def attend(q, pool, table, block_pos, n, tail, scale, cap=0.0, slopes=None, prefix=0, doc_start=0,
           window=0, n_pages=None):
    """One sequence. q [H][d], pool [pages][2][Hkv][64][d] (float64), table / block_pos rows.
    Returns out [H][d], mass [n] (each entry's weight over all heads), and two arrays that error
    bounds need: the weighted sum of |V| per output, and the largest sum of |q k| per head."""
    H, d = q.shape
    Hkv = pool.shape[2]
    G = H // Hkv
    out, absv, big = np.zeros((H, d)), np.zeros((H, d)), np.zeros(H)
    mass = np.zeros(max(n, 0))
    if n <= 0:
        return out, mass, absv, big
    pos, x_b = seen_positions(block_pos, n, tail, prefix, doc_start, window)
    pages = len(pool) if n_pages is None else n_pages
    pos = [p for p in pos if 0 <= int(table[p[0]]) < pages]
    if not pos:
        return out, mass, absv, big
    ent = np.array([p[0] for p in pos])
    slot = np.array([p[1] for p in pos])
    at = np.array([p[2] for p in pos], dtype=np.float64)
    page = np.asarray(table)[ent]
    for h in range(H):
        if h % G == 0:
            K, V = pool[page, 0, h // G, slot], pool[page, 1, h // G, slot]
            aK, aV = np.abs(K), np.abs(V)
        z = scale * (K @ q[h])
        if cap > 0:
            z = cap * np.tanh(z / cap)
        if slopes is not None:
            z = z - slopes[h] * (x_b - at)
        w = np.exp(z - z.max())
        w = w / w.sum()
        out[h] = w @ V
        absv[h] = w @ aV
        big[h] = scale * (aK @ np.abs(q[h])).max()
        mass += np.bincount(ent, weights=w, minlength=n)
    return out, mass, absv, big


def append(n, tail, free, cnt, table, block_pos, bt_stride):
    """`cnt` tokens behind a sequence of n entries. Returns (n, tail, free, [(page, slot)] of the
    tokens, {entry: (page, position)} opened), or None where pages or entries do not suffice."""
    free = list(free)
    dest, opened = [], {}
    table, pos = dict(enumerate(table[:n])), dict(enumerate(block_pos[:n]))
    for _ in range(cnt):
        if n == 0 or tail == PAGE:
            if not free or n >= bt_stride:
                return None
            page = free.pop()
            pos[n] = pos[n - 1] + 1 if n > 0 else 0
            table[n] = page
            opened[n] = (page, pos[n])
            n, tail = n + 1, 0
        dest.append((table[n - 1], tail))
        tail += 1
    return n, tail, free, dest, opened


def evict(score, n, budget, n_sink, n_recent):
    """Kept and freed entries of one sequence, both ascending."""
    if n <= budget:
        return list(range(n)), []
    middle = list(range(n_sink, n - n_recent))
    rank = sorted(middle, key=lambda j: (-np.inf if np.isnan(score[j]) else score[j], -j), reverse=True)
    # NaN ranks below -inf
    rank = [j for j in rank if not np.isnan(score[j])] + [j for j in middle if np.isnan(score[j])]
    best = set(rank[:budget - n_sink - n_recent])
    kept = [j for j in range(n) if j < n_sink or j >= n - n_recent or j in best]
    return kept, [j for j in range(n) if j not in set(kept)]
