"""Plain float64 oracle of the paged latent cache and of sampling under filters (test
infrastructure; shares no code with the library).

The cache's row of position j of sequence b is row j % page of page table[b][j // page]. Pages
that are free lie on one stack, its top the last of the first n_free entries.
"""
from __future__ import annotations

import math

import numpy as np


def page_assign(table, held, free, n_free, new_len, page, start=None, T=0):
    """Lists and arrays in, (table, held, free, n_free, slots or None, err) out, from the words of the contract."""
    table, held, free = table.copy(), held.copy(), free.copy()
    B, W = table.shape
    need = [-(-int(n) // page) for n in new_len]
    sound = [0 <= int(new_len[b]) and need[b] <= W and 0 <= held[b] <= W for b in range(B)]
    given = [int(table[b, k]) for b in range(B) if sound[b] for k in range(need[b], held[b])]
    stack = free[:n_free].tolist() + given[::-1]
    room, asked, refused = len(stack), 0, []
    for b in range(B):
        if not sound[b]:
            refused.append(b)
            continue
        miss = max(need[b] - int(held[b]), 0)
        asked += miss
        if miss and asked > room:
            refused.append(b)
            continue
        for k in range(int(held[b]), need[b]):
            table[b, k] = stack.pop()
        held[b] = need[b]
    out = free.copy()
    out[:len(stack)] = stack
    slots = None
    if T:
        slots = np.full((B, T), -1, dtype=np.int32)
        for b in range(B):
            for i in range(T):
                j = int(start[b]) + i
                if b not in refused and 0 <= j < new_len[b]:
                    slots[b, i] = table[b, j // page] * page + j % page
    return table, held, out, len(stack), slots, (refused[0] + 1 if refused else 0)


def rows_of(table_row, n, page):
    """Cache rows of positions 0 .. n - 1."""
    j = np.arange(n)
    return table_row[j // page].astype(np.int64) * page + j % page


def sample(logits, u, temperature, top_k, top_p, min_p):
    """One row in float64: (token, log-probability, the draw's distance to the nearest border over the kept mass)."""
    l = logits.astype(np.float64)
    if temperature == 0:
        return int(np.argmax(l)), 0.0, 1.0
    y = (l - l.max()) / temperature
    w = np.rint(np.exp(y) * 2.0 ** 44).astype(np.int64)
    order = np.lexsort((np.arange(len(l)), -l))
    if 0 < top_k < len(l):
        order = order[:top_k]
    near = 1.0
    if top_p < 1.0:
        mass = np.cumsum(w[order])
        goal = top_p * float(mass[-1])
        n = int((mass.astype(np.float64) < goal).sum()) + 1
        near = float(np.abs(mass - goal).min()) / float(mass[-1])
        order = order[:n]
    order = order[w[order] >= min(max(min_p, 0.0), 1.0) * 2.0 ** 44]
    keep = np.sort(order)
    up = np.cumsum(w[keep])
    t = float(u) * float(up[-1])
    k = min(int((up.astype(np.float64) <= t).sum()), len(keep) - 1)
    near = min(near, float(np.abs(up[:-1] - t).min()) / float(up[-1])) if len(keep) > 1 else near
    return int(keep[k]), float(y[keep[k]] - math.log(float(w.astype(np.float64).sum()) / 2.0 ** 44)), near
