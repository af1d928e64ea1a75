"""Oracle of the pages' coming and going (include/paged_pages.h): one row and page at a time, in
numpy, without any code of the library.  The inputs are left as they are."""
from __future__ import annotations

import numpy as np


def _ring(free_pages, state):
    P = len(free_pages)
    return int(state[0]) % P, min(max(int(state[1]), 0), P)


def fork(parents, children, table, kv_lens, holders, free_pages, free_state, page_size, table_out, kv_lens_out):
    """Returns (table, kv_lens, holders, moves, free_state) after the fork; table_out and kv_lens_out are what
    the outputs held before."""
    N, width = table.shape
    P = len(free_pages)
    head, count = _ring(free_pages, free_state)
    out, lens, held = np.array(table_out), np.array(kv_lens_out), np.array(holders)
    moves = np.full((len(parents), 2), -1, np.int32)
    taken = wanted = 0
    for i, (p, c) in enumerate(zip(parents, children)):
        if not (0 <= p < N and 0 <= c < N):
            continue
        L = max(int(kv_lens[p]), 0)
        lens[c] = L
        full = min(L // page_size, width)
        for j in range(full):
            out[c, j] = table[p, j]
            if 0 <= table[p, j] < P:
                held[table[p, j]] += 1
        if L % page_size and full < width:
            wanted += 1
            f = -1
            if taken < count:
                f = int(free_pages[(head + taken) % P])
                taken += 1
            out[c, full] = f
            if 0 <= f < P and 0 <= table[p, full] < P:
                moves[i] = table[p, full], f
    state = np.array([(head + taken) % P, count - taken, wanted - taken], np.int32)
    return out, lens, held, moves, state


def release(first, end, table, holders, free_pages, free_state, table_out):
    """Returns (table, holders, free_pages, free_state)."""
    N, width = table.shape
    P = len(free_pages)
    head, count = _ring(free_pages, free_state)
    out, held, ring = np.array(table_out), np.array(holders), np.array(free_pages)
    gone = {}
    for n in range(N):
        for j in range(max(int(first[n]), 0), min(int(end[n]), width)):
            out[n, j] = -1
            p = int(table[n, j])
            if 0 <= p < P:
                gone[p] = gone.get(p, 0) + 1
    freed = 0
    for p in sorted(gone):
        if gone[p] > held[p]:
            ring[(head + count + freed) % P] = p
            freed += 1
        held[p] = max(0, held[p] - gone[p])
    return out, held, ring, np.array([head, min(count + freed, P), 0], np.int32)


def compact(kv_lens, table, holders, free_pages, page_size):
    """Returns (table, holders, free_pages, free_state, moves)."""
    N, width = table.shape
    P = len(holders)
    at = [(n, j) for n in range(N) for j in range(min(-(-max(int(kv_lens[n]), 0) // page_size), width))
          if 0 <= table[n, j] < P]
    used = sorted({int(table[x]) for x in at})
    U = len(used)
    to = {p: p for p in used if p < U}
    pairs = list(zip([p for p in used if p >= U], sorted(set(range(U)) - set(used))))
    to.update(pairs)
    out, held, ring = np.array(table), np.zeros_like(holders), np.array(free_pages)
    for x in at:
        out[x] = to[int(table[x])]
    for p in used:
        held[to[p]] = holders[p]
    ring[:P - U] = np.arange(U, P)
    moves = np.full((P // 2, 2), -1, np.int32)
    if pairs:
        moves[:len(pairs)] = pairs
    return out, held, ring, np.array([0, P - U, 0], np.int32), moves


def copy(cache, moves):
    """cache [P, ...] with its pages moved."""
    out = np.array(cache)
    for a, b in moves:
        if 0 <= a < len(cache) and 0 <= b < len(cache):
            out[b] = cache[a]
    return out
