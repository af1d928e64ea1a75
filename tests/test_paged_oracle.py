"""Pins of the paged-cache oracle (CPU): closed forms, invariants and counting arguments that do
not depend on how the oracle computes."""
import numpy as np

from oracle import paged as O


def cache_of(K, s, rng, spare=3):
    """K [n, H, D] laid into scattered pages of s slots: (cache with NaN elsewhere, table row)."""
    n, H, D = K.shape
    used = -(-n // s)
    cache = np.full((used + spare, s, H, D), np.nan)
    ids = rng.permutation(used + spare)[:used]
    for j in range(n):
        cache[ids[j // s], j % s] = K[j]
    return cache, ids.astype(np.int32)[None, :]


def test_one_key_returns_its_value_and_equal_keys_the_mean():
    rng = np.random.default_rng(0)
    V = rng.standard_normal((5, 1, 8))
    K = np.ones((5, 1, 8)) * 0.3
    kc, table = cache_of(K, 4, rng)
    vc = np.full_like(kc, np.nan)
    for j in range(5):
        vc[table[0, j // 4], j % 4] = V[j]
    q = rng.standard_normal((5, 2, 8))
    o, lse, _, _ = O.attention(q, kc, vc, table, np.array([0, 5]), np.array([5]), 0.5)
    for i in range(5):   # token i sees i + 1 equal keys
        np.testing.assert_allclose(o[i], np.broadcast_to(V[:i + 1, 0].mean(0), (2, 8)), rtol=1e-13)
        np.testing.assert_allclose(lse[i], 0.5 * 0.3 * q[i].sum(-1) + np.log(i + 1), rtol=1e-12)


def test_window_and_chunks_agree_with_whole_and_with_cut_caches():
    rng = np.random.default_rng(1)
    n, H, D = 23, 2, 8
    K, V = rng.standard_normal((n, H, D)), rng.standard_normal((n, H, D))
    kc, table = cache_of(K, 8, rng)
    vc = np.full_like(kc, np.nan)
    for j in range(n):
        vc[table[0, j // 8], j % 8] = V[j]
    q = rng.standard_normal((n, 4, D))
    whole, lw, _, _ = O.attention(q, kc, vc, table, np.array([0, n]), np.array([n]), 0.3, window=5)
    # the last 7 tokens as a chunk of their own
    part, lp, _, _ = O.attention(q[-7:], kc, vc, table, np.array([0, 7]), np.array([n]), 0.3, window=5)
    np.testing.assert_allclose(part, whole[-7:], rtol=1e-13)
    np.testing.assert_allclose(lp, lw[-7:], rtol=1e-13)
    # a window of 5 is a cache of 5
    kc5, t5 = cache_of(K[-5:], 8, rng)
    vc5 = np.full_like(kc5, np.nan)
    vc5[t5[0, 0], :5] = V[-5:]
    one, lo, _, _ = O.attention(q[-1:], kc5, vc5, t5, np.array([0, 1]), np.array([5]), 0.3)
    np.testing.assert_allclose(one[0], whole[-1], rtol=1e-13)
    np.testing.assert_allclose(lo[0], lw[-1], rtol=1e-13)


def test_split_keys_join_by_their_lse():
    """Softmax over a union of keys from the softmaxes over its parts: the weights are
    exp(lse_part - lse)."""
    rng = np.random.default_rng(2)
    n, D = 20, 8
    K, V = rng.standard_normal((n, 1, D)), rng.standard_normal((n, 1, D))
    q = rng.standard_normal((1, 3, D))

    def run(sl):
        kc, t = cache_of(K[sl], 8, rng)
        vc = np.full_like(kc, np.nan)
        for j, x in enumerate(V[sl]):
            vc[t[0, j // 8], j % 8] = x
        m = len(K[sl])
        o, lse, _, _ = O.attention(q, kc, vc, t, np.array([0, 1]), np.array([m]), 0.7)
        return o[0], lse[0]
    o, L = run(slice(0, n))
    a, La = run(slice(0, 9))
    b, Lb = run(slice(9, n))
    np.testing.assert_allclose(np.logaddexp(La, Lb), L, rtol=1e-13)
    np.testing.assert_allclose(np.exp(La - L)[:, None] * a + np.exp(Lb - L)[:, None] * b, o, rtol=1e-12)


def test_rows_without_keys():
    q = np.ones((3, 1, 8))
    kc = np.full((2, 8, 1, 8), np.nan)
    kc[0, 0] = 1.0
    o, lse, _, _ = O.attention(q, kc, kc, np.array([[0]], np.int32), np.array([0, 3]), np.array([1]), 1.0)
    assert np.all(o[:2] == 0) and np.all(lse[:2] == -np.inf)
    assert np.all(o[2] == 1) and np.isfinite(lse[2]).all()


def test_plan_counts_pages_and_gives_every_token_its_own_slot():
    rng = np.random.default_rng(3)
    s, N, P, width = 8, 6, 40, 7
    cached, new = np.array([0, 5, 8, 16, 3, 20]), np.array([9, 3, 0, 1, 14, 4])
    held = -(-cached // s)
    ids = rng.permutation(P)
    table = np.full((N, width), 99)
    used = 0
    for n in range(N):
        table[n, :held[n]] = ids[used:used + held[n]]
        used += held[n]
    free = np.zeros(P, np.int32)
    head, count = 37, P - used
    for i in range(count):
        free[(head + i) % P] = ids[used + i]
    t2, cu, kv, pos, slots, st = O.plan(cached, new, free, [head, count, 0], table, s, 33)
    need = int((-(-(cached + new) // s) - held).sum())
    assert list(st) == [(head + need) % P, count - need, 0]
    assert list(cu) == [0, 9, 12, 12, 13, 27, 31] and list(kv) == list(cached + new)
    live = slots[:31]
    assert len(set(live)) == 31 and live.min() >= 0 and list(slots[31:]) == [-1, -1]
    # no two requests share a page, and a token's slot lies in its request's page at its offset
    owned = [set(t2[n, :-(-int(kv[n]) // s)]) for n in range(N)]
    assert sum(map(len, owned)) == len(set().union(*owned)) == used + need
    for n in range(N):
        for t in range(cu[n], cu[n + 1]):
            assert slots[t] // s == t2[n, pos[t] // s] and slots[t] % s == pos[t] % s
            assert pos[t] == cached[n] + t - cu[n]


def test_plan_without_enough_pages():
    free = np.array([4, 5, 6, 7], np.int32)
    t, cu, kv, pos, slots, st = O.plan([0, 0], [20, 20], free, [3, 3, 0], np.zeros((2, 3), np.int32), 8, 40)
    assert list(st) == [2, 0, 3]                       # six pages wanted, three had
    assert list(t[0]) == [7, 4, 5] and list(t[1]) == [-1, -1, -1]
    assert list(slots[20:]) == [-1] * 20 and slots[0] == 56
    # a table two pages wide: the third page of each is past it
    t, _, _, _, slots, st = O.plan([0, 0], [20, 20], free, [0, 4, 0], np.zeros((2, 2), np.int32), 8, 40)
    assert list(st) == [0, 0, 2] and list(slots[16:20]) == [-1] * 4 and slots[20] >= 0


def test_write_puts_rows_in_their_slots():
    rng = np.random.default_rng(4)
    cache = rng.standard_normal((3, 8, 2, 4))
    rows = rng.standard_normal((4, 2, 4))
    out = O.write(cache, rows, [5, -1, 23, 24])
    np.testing.assert_array_equal(out[0, 5], rows[0])
    np.testing.assert_array_equal(out[2, 7], rows[2])
    out[0, 5], out[2, 7] = cache[0, 5], cache[2, 7]
    np.testing.assert_array_equal(out, cache)
