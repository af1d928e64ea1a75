"""Float64 oracle of the paged cache (include/paged_attn.h): the plan of a step, the write, and
the attention, one request, token and head at a time, in numpy, without any code of the library.
"""
from __future__ import annotations

import numpy as np


def plan(cached, new, free_pages, free_state, table, page_size, tokens):
    """Returns (table, cu, kv_lens, positions, slots, free_state) after the step; the inputs are
    left as they are."""
    table = np.array(table)
    N, width = table.shape
    P = len(free_pages)
    head, count = int(free_state[0]) % P, min(max(int(free_state[1]), 0), P)
    ring = [int(free_pages[(head + i) % P]) for i in range(count)]
    cu, kv_lens, short, taken = [0], [], 0, 0
    positions, slots = np.zeros(tokens, np.int32), np.full(tokens, -1, np.int64)
    for n in range(N):
        c, q = max(int(cached[n]), 0), max(int(new[n]), 0)
        for p in range(-(-c // page_size), -(-(c + q) // page_size)):
            if p >= width:
                short += 1
            elif taken < count:
                table[n, p] = ring[taken]
                taken += 1
            else:
                table[n, p] = -1
                short += 1
        for i in range(q):
            t, pos = cu[-1] + i, c + i
            if t < tokens:
                positions[t] = pos
                p = pos // page_size
                if p < width and table[n, p] >= 0:
                    slots[t] = int(table[n, p]) * page_size + pos % page_size
        cu.append(cu[-1] + q)
        kv_lens.append(c + q)
    state = np.array([(head + taken) % P, count - taken, short], np.int32)
    return table, np.array(cu, np.int32), np.array(kv_lens, np.int32), positions, slots, state


def write(cache, rows, slots):
    """cache [P, s, H, D] with rows [T, H, D] in their slots."""
    cache = np.array(cache)
    P, s = cache.shape[:2]
    for t, slot in enumerate(slots):
        if 0 <= slot < P * s:
            cache[slot // s, slot % s] = rows[t]
    return cache


def attention(q, k_cache, v_cache, table, cu, kv_lens, scale, window=0):
    """o [T, Hq, D], lse [T, Hq], and two magnitudes for error bounds: the weighted mean of |v|
    [T, Hq, D] and the largest sum of |scale q_d k_jd| over the keys seen [T, Hq].  Rows of no
    request stay NaN."""
    T, Hq, D = q.shape
    P, s, Hkv, _ = k_cache.shape
    g = Hq // Hkv
    o = np.full((T, Hq, D), np.nan)
    av = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    qk = np.full((T, Hq), np.nan)
    for n in range(len(kv_lens)):
        first, new, kv = int(cu[n]), int(cu[n + 1]) - int(cu[n]), int(kv_lens[n])
        j = np.arange(max(kv, 0))
        ids = table[n, np.minimum(j // s, table.shape[1] - 1)].astype(np.int64) if kv else j
        bad = (ids < 0) | (ids >= P) | (j // s >= table.shape[1])
        ids = np.where(bad, 0, ids)
        for h in range(Hkv):
            K, V = k_cache[ids, j % s, h], v_cache[ids, j % s, h]
            K, V = np.where(bad[:, None], 0.0, K), np.where(bad[:, None], 0.0, V)
            for i in range(new):
                p = kv - new + i
                lo = max(0, p - window + 1) if window else 0
                r, hs = first + i, slice(h * g, (h + 1) * g)
                if p < 0:
                    o[r, hs], av[r, hs], lse[r, hs], qk[r, hs] = 0.0, 0.0, -np.inf, 0.0
                    continue
                Kv, Vv = K[lo:p + 1], V[lo:p + 1]
                S = scale * (q[r, hs] @ Kv.T)
                m = S.max(axis=1, keepdims=True)
                e = np.exp(S - m)
                l = e.sum(axis=1, keepdims=True)
                o[r, hs] = (e / l) @ Vv
                av[r, hs] = (e / l) @ np.abs(Vv)
                lse[r, hs] = (m + np.log(l))[:, 0]
                qk[r, hs] = (scale * (np.abs(q[r, hs]) @ np.abs(Kv).T)).max(axis=1)
    return o, lse, av, qk
