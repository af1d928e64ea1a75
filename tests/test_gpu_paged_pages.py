"""GPU parity of the calls on a cache's pages (include/paged_pages.h) with their oracle: whole numbers and
copies, all equal.  And what they do together with the plan, the write and the attention."""
import numpy as np
import pytest
import torch

from oracle import paged_pages as O
from linear_recurrent_rnn_gb300 import librglru as R
from test_gpu_paged import DT, compare, expect, f64

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def pool(rng, N, most, s, spare, share=0.0):
    """N rows of up to `most` tokens in scattered pages, some pages with more holders, stale entries behind:
    (table, lens, holders, ring, state)."""
    lens = rng.integers(0, most + 1, N)
    held = -(-lens // s)
    width = most // s + 3
    P = int(held.sum()) + spare
    ids = rng.permutation(P)
    table = rng.choice([-1, 0, P - 1, P, 2 ** 30], size=(N, width))
    at = 0
    for n in range(N):
        table[n, :held[n]] = ids[at:at + held[n]]
        at += held[n]
    holders = np.zeros(P, np.int64)
    holders[ids[:at]] = (rng.random(at) < share) * rng.integers(1, 3, at)
    ring, head = np.full(P, -1, np.int64), int(rng.integers(0, P))
    ring[(head + np.arange(P - at)) % P] = ids[at:]
    return table, lens, holders, ring, [head, P - at, 0]


def check(got, want, names):
    for n, a, b in zip(names, got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b, err_msg=n)


# ---------------------------------------------------------------- fork
def run_fork(parents, children, table, lens, holders, ring, state, s, table_out, lens_out, in_place):
    N, width = table.shape
    sh = R.make_paged_shape(N, 0, num_pages=len(ring), page_size=s, table_width=width)
    t, L, h, st = i32(table), i32(lens), i32(holders), i32(state)
    to, lo, ho, so = (t, L, h, st) if in_place else (i32(table_out), i32(lens_out), torch.full_like(h, 7), torch.full_like(st, 7))
    moves = torch.full((len(parents), 2), 7, dtype=torch.int32, device="cuda")
    R.paged_fork(sh, i32(parents), i32(children), t, L, h, i32(ring), st, to, lo, ho, moves, so)
    return to, lo, ho, moves, so


FORK_OUT = ("table", "lens", "holders", "moves", "state")
FORKS = {  # rows, most tokens, page, children, spare pages
    "one": (2, 40, 16, 1, 5), "four": (6, 500, 8, 4, 9), "many": (700, 300, 16, 600, 700), "wide": (40, 16000, 16, 30, 40),
    "pages-run-out": (30, 200, 16, 20, 6), "none-free": (9, 90, 32, 4, 0), "most": (8192, 20, 8, 4096, 5000),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(FORKS))
def test_fork_matches_oracle(name, in_place):
    N, most, s, M, spare = FORKS[name]
    rng = np.random.default_rng(N + M)
    table, lens, holders, ring, state = pool(rng, N, most, s, max(spare, 1), 0.3)
    if spare == 0:
        state[1] = 0
    rows = rng.permutation(N)
    children, parents = rows[:M], rng.choice(rows[M:], M)
    lens[parents[0]] = min(most, 2 * s)  # a whole number of pages
    to, lo = (table, lens) if in_place else (rng.integers(-1, 9, table.shape), rng.integers(0, 9, N))
    want = O.fork(parents, children, table, lens, holders, ring, state, s, to, lo)
    check(run_fork(parents, children, table, lens, holders, ring, state, s, to, lo, in_place), want, FORK_OUT)


def test_a_step_of_a_beam_forks_every_row_from_any():
    """Into a second table every row may be child and parent; the first table's rows are released after."""
    rng = np.random.default_rng(3)
    N, s = 24, 16
    table, lens, holders, ring, state = pool(rng, N, 300, s, 60)
    parents = rng.integers(0, N, N)
    zeros = np.zeros_like(table)
    want = O.fork(parents, np.arange(N), table, lens, holders, ring, state, s, zeros, lens * 0)
    got = run_fork(parents, np.arange(N), table, lens, holders, ring, state, s, zeros, lens * 0, False)
    check(got, want, FORK_OUT)
    end = -(-lens // s)
    want2 = O.release(lens * 0, end, table, want[2], ring, want[4], table)
    got2 = run_release(lens * 0, end, table, got[2].cpu().numpy(), ring, want[4], True)
    check(got2, want2, RELEASE_OUT)
    # what is free and what the new rows hold are all the pages, each once
    free = [int(want2[2][(want2[3][0] + i) % len(ring)]) for i in range(want2[3][1])]
    used = {int(got[0][n, j]) for n in range(N) for j in range(-(-int(want[1][n]) // s))}
    assert sorted(free + list(used)) == list(range(len(ring)))


def test_fork_passes_over_what_is_out_of_range():
    rng = np.random.default_rng(5)
    table, lens, holders, ring, state = pool(rng, 8, 100, 16, 20)
    table[2, :3], lens[2], lens[3], lens[4] = [-1, len(ring), 2 ** 30], 55, -7, 2 ** 30
    ring[(state[0] + 1) % len(ring)] = 2 ** 30  # no page
    for st in (state, [state[0] - 3 * len(ring), 10 ** 6, 5], [state[0], -4, 0]):
        args = ([0, 9, -1, 2, 3, 4, 2], [5, 6, 6, 7, 0, 1, 6], table, lens, holders, ring, st, 16, table * 0, lens * 0)
        check(run_fork(*args, False), O.fork(*args), FORK_OUT)


def test_no_children():
    rng = np.random.default_rng(6)
    table, lens, holders, ring, state = pool(rng, 3, 60, 8, 5)
    args = ([], [], table, lens, holders, ring, state, 8, table, lens)
    check(run_fork(*args, False), O.fork(*args), FORK_OUT)


# ---------------------------------------------------------------- release
RELEASE_OUT = ("table", "holders", "ring", "state")


def run_release(first, end, table, holders, ring, state, in_place, ws=None, table_out=None):
    N, width = table.shape
    sh = R.make_paged_shape(N, 0, num_pages=len(ring), page_size=16, table_width=width)
    ws = R.alloc_paged_pages_workspace(sh) if ws is None else ws
    t, h, st, r = i32(table), i32(holders), i32(state), i32(ring)
    to, ho, so = (t, h, st) if in_place else (i32(table if table_out is None else table_out), torch.full_like(h, 7), torch.full_like(st, 7))
    R.paged_release(sh, i32(first), i32(end), t, h, r, st, to, ho, so, ws)
    assert not ws[:256 + 4 * (-(-len(ring) // 32))].any()
    return to, ho, r, so


RELEASES = {"one": (1, 40, 3), "some": (9, 500, 9), "many": (600, 3000, 77), "long": (3, 200000, 5), "small-pool": (2, 20, 1)}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(RELEASES))
def test_release_matches_oracle(name, in_place):
    N, most, spare = RELEASES[name]
    rng = np.random.default_rng(N + most)
    table, lens, holders, ring, state = pool(rng, N, most, 16, spare, 0.4)
    held = -(-lens // 16)
    first = rng.integers(0, held + 1) * (rng.random(N) < 0.5)
    end = np.where(rng.random(N) < 0.7, held, rng.integers(first, held + 1))
    out = table if in_place else rng.integers(0, 9, table.shape)
    want = O.release(first, end, table, holders, ring, state, out)
    check(run_release(first, end, table, holders, ring, state, in_place, table_out=out), want, RELEASE_OUT)


def test_pages_of_several_rows_go_with_the_last():
    """A prompt's pages in five rows: released row by row, in one call or in several."""
    table = np.array([[3, 7, 9, -1]] * 5)
    table[:, 2] = [9, 10, 11, 12, 13]
    holders = np.zeros(20, np.int64)
    holders[[3, 7]] = 4
    ring, state = np.full(20, 19), [18, 3, 0]
    end = [3] * 5
    want = O.release([0] * 5, end, table, holders, ring, state, table)
    assert list(want[3]) == [18, 10, 0]
    check(run_release([0] * 5, end, table, holders, ring, state, True), want, RELEASE_OUT)
    for ends in ([3, 0, 0, 0, 0], [0, 3, 3, 0, 0], [0, 0, 0, 3, 3]):
        want = O.release([0] * 5, ends, table, holders, ring, state, table)
        check(run_release([0] * 5, ends, table, holders, ring, state, True), want, RELEASE_OUT)
        table, holders, ring, state = (np.array(w) for w in want)
    assert list(state) == [18, 10, 0] and not holders.any()


def test_release_of_what_is_out_of_range_or_released():
    """Ranges past the table, negative and empty ones; entries that are no pages; the same page twice; holders
    that are negative; a ring said to be over-full."""
    table = np.array([[0, 1, -1, 2 ** 30], [1, 1, 4, 5], [6, 7, 8, 9], [4, 4, 4, 4]])
    holders = np.zeros(11, np.int64)
    holders[[4, 5, 6]] = [2, -3, 1]
    for state in ([0, 1, 0], [-1, 11, 3], [40, 99, 0], [3, -5, 0]):
        args = ([-5, 0, 3, 1], [9, 4, 1, 2 ** 30], table, holders, np.arange(11), state)
        want = O.release(*args, table)
        for in_place in (False, True):
            check(run_release(*args, in_place), want, RELEASE_OUT)
    again = run_release([0] * 4, [4] * 4, np.full((4, 4), -1), holders * 0, np.arange(11), [2, 5, 0], True)
    assert again[3].tolist() == [2, 5, 0] and again[2].tolist() == list(range(11))


# ---------------------------------------------------------------- compact
COMPACT_OUT = ("table", "holders", "ring", "state", "moves")


def run_compact(lens, table, holders, ring, s, in_place, ws=None):
    N, width = table.shape
    P = len(ring)
    sh = R.make_paged_shape(N, 0, num_pages=P, page_size=s, table_width=width)
    ws = R.alloc_paged_pages_workspace(sh) if ws is None else ws
    t, h, r = i32(table), i32(holders), i32(ring)
    to, ho = (t, h) if in_place else (torch.full_like(t, 7), torch.full_like(h, 7))
    st, moves = torch.full((3,), 7, dtype=torch.int32, device="cuda"), torch.full((P // 2, 2), 7, dtype=torch.int32, device="cuda")
    R.paged_compact(sh, i32(lens), t, h, to, ho, r, st, moves, ws)
    assert not ws[:256 + 4 * (-(-P // 32))].any()
    return to, ho, r, st, moves


COMPACTS = {"one": (1, 40, 16, 1), "few": (7, 200, 8, 300), "half": (90, 900, 16, 3000), "full": (30, 400, 16, 0),
            "many": (900, 2000, 16, 40000), "nearly-empty": (2, 60, 16, 5000), "odd": (5, 77, 32, 31)}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(COMPACTS))
def test_compact_matches_oracle(name, in_place):
    N, most, s, spare = COMPACTS[name]
    rng = np.random.default_rng(N + most)
    table, lens, holders, ring, _ = pool(rng, N, most, s, spare + (1 if name == "one" else 0), 0.3)
    if N > 5:  # shared pages, a row without tokens, one longer than the table
        table[3, :5], lens[3], lens[4] = table[2, :5], min(lens[2], 5 * s), 0
        lens[5] = 2 ** 30
        table[5] = -1
    if len(ring) == 0:
        return
    want = O.compact(lens, table, holders, ring, s)
    check(run_compact(lens, table, holders, ring, s, in_place), want, COMPACT_OUT)


def test_nothing_in_use_and_a_pool_of_one_page():
    for P in (1, 2, 33):
        for lens in ([0], [3], [-1]):
            args = (np.array(lens), np.array([[P - 1, 5]]), np.ones(P, np.int64), np.arange(P))
            check(run_compact(*args, 8, False), O.compact(*args, 8), COMPACT_OUT)


# ---------------------------------------------------------------- copy
def test_copy_of_caches_of_any_kind():
    """Types, layouts, pages of odd sizes, a page within a larger block; moves that are none."""
    P, s = 37, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *z: torch.randn(*z, generator=g, device="cuda")
    caches = [r(P, s, 2, 64).bfloat16(), r(P, s, 3, 40), r(P, 2, s, 64).bfloat16().transpose(1, 2),
              r(P, 2, s, 2, 64).bfloat16()[:, 1], (r(P, s, 1, 5) * 9).to(torch.uint8), r(P, 3)[:, :1],
              r(P, 4, s, 48).bfloat16()[..., :40].transpose(1, 2), r(P, s * 3000), r(P * 3 + 1)[1:].view(P, 3)]
    moves = np.array([[0, 36], [5, 4], [-1, -1], [7, P], [-3, 8], [11, 12], [2 ** 30, 1], [35, 20], [13, 21]])
    want = [O.copy(c.double().cpu().numpy(), moves) for c in caches]
    R.paged_copy(R.make_paged_shape(1, 0, num_pages=P, page_size=s, table_width=1), i32(moves), *caches)
    for c, w in zip(caches, want):
        np.testing.assert_array_equal(f64(c), w)


def test_copy_leaves_the_neighbours():
    """Bytes of a cache's last page are the last ones that are touched; a block's other parts keep their values."""
    P = 5
    block = torch.arange(P * 3 * 7 + 9, dtype=torch.uint8, device="cuda")
    part = block[:P * 21].view(P, 3, 7)[:, 1]
    want = block.clone()
    want[:P * 21].view(P, 3, 7)[4, 1] = part[0]
    R.paged_copy(R.make_paged_shape(1, 0, num_pages=P, page_size=8, table_width=1), i32([[0, 4]]), part)
    assert torch.equal(block, want)


def test_copy_of_many_caches_and_none():
    caches = [torch.full((3, 4), float(c), device="cuda") for c in range(131)]
    for c in caches:
        c[2] = -1
    sh = R.make_paged_shape(1, 0, num_pages=3, page_size=8, table_width=1)
    before = R.rglru_kernel_launches()
    R.paged_copy(sh, i32([[2, 0]]), *caches)
    assert R.rglru_kernel_launches() == before + 3  # 64 caches a launch
    assert all(bool((c[0] == -1).all() and (c[1] == k).all()) for k, c in enumerate(caches))
    R.paged_copy(sh, i32([[2, 0]]))
    R.paged_copy(sh, i32(np.zeros((0, 2))), *caches)
    assert R.rglru_kernel_launches() == before + 3


def test_copy_where_offsets_pass_32_bits():
    P = 4200
    c = torch.zeros(P, 2 ** 20, dtype=torch.uint8, device="cuda")
    c[1] = torch.randint(1, 255, (2 ** 20,), dtype=torch.uint8, device="cuda")
    R.paged_copy(R.make_paged_shape(1, 0, num_pages=P, page_size=8, table_width=1), i32([[1, P - 1], [P - 2, 0]]), c)
    assert torch.equal(c[P - 1], c[1]) and not c[P - 2].any() and not c[0].any()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_requests_fork_go_on_end_and_the_pool_is_closed_up(io):
    """A prompt, answers that fork from it and from one another, some that end, the pool closed up, and all go
    on: every request's attention is that over its own tokens.  All steps of the pages come from graphs that are
    captured once and replayed."""
    dt, Hq, Hkv, D, s, width, P, N = DT[io], 4, 2, 64, 8, 12, 70, 6
    z = lambda *n, dtype=torch.int32: torch.zeros(*n, dtype=dtype, device="cuda")
    lens, new, holders, state = z(N), z(N), z(P), i32([9, P, 0])
    ring = i32(np.random.default_rng(1).permutation(P))
    table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((P, s, Hkv, D), float("nan"), dtype=dt, device="cuda") for _ in range(2))
    T = 45
    cu, pos, slots, lse = z(N + 1), z(T), z(T, dtype=torch.int64), z(T, Hq, dtype=torch.float32)
    q, o = z(T, Hq, D, dtype=dt), z(T, Hq, D, dtype=dt)
    k, v = z(T, Hkv, D, dtype=dt), z(T, Hkv, D, dtype=dt)
    sh = R.make_paged_shape(N, T, Hq, Hkv, D, P, s, width, io=dt)
    ws, pages_ws = R.alloc_paged_workspace(sh), R.alloc_paged_pages_workspace(sh)
    parents, children, moves = i32([-1, -1]), i32([-1, -1]), z(2, 2)
    first, end, all_moves = z(N), z(N), z(P // 2, 2)

    def step():
        R.paged_plan(sh, lens, new, ring, state, table, cu, lens, pos, slots, state)
        R.paged_kv_write(sh, k, v, slots, kc, vc)
        R.paged_attention(sh, q, kc, vc, table, cu, lens, 0.125, o, lse, ws)

    def fork():
        R.paged_fork(sh, parents, children, table, lens, holders, ring, state, table, lens, holders, moves, state)
        R.paged_copy(sh, moves, kc, vc)

    def release():
        R.paged_release(sh, first, end, table, holders, ring, state, table, holders, state, pages_ws)

    def compact():
        R.paged_compact(sh, lens, table, holders, table, holders, ring, state, all_moves, pages_ws)
        R.paged_copy(sh, all_moves, kc, vc)

    graphs = {}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f in (step, fork, release, compact):
            f()  # warm-up: nothing new, no children, nothing released, nothing in use
    torch.cuda.current_stream().wait_stream(side)
    for f in (step, fork, release, compact):
        graphs[f] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[f]):
            f()

    rng = np.random.default_rng(2)
    seqs = [[np.zeros((0, h, D)) for h in (Hkv, Hkv)] for _ in range(N)]

    def append(news):
        new.copy_(i32(news))
        for t, H in ((q, Hq), (k, Hkv), (v, Hkv)):
            t.copy_(torch.from_numpy(rng.standard_normal((T, H, D))))
        graphs[step].replay()
        at = 0
        for n, m in enumerate(news):
            for i, t in enumerate((k, v)):
                seqs[n][i] = np.concatenate([seqs[n][i], f64(t)[at:at + m]])
            if m:
                L = len(seqs[n][0])
                x = dict(q=q[at:at + m], kc=torch.from_numpy(seqs[n][0][None]), vc=torch.from_numpy(seqs[n][1][None]),
                         table=i32([[0]]), cu=i32([0, m]), kv=i32([L]))
                compare(o[at:at + m], lse[at:at + m], expect(x, 0.125), io)
            at += m
        assert int(state[2]) == 0

    def do_fork(pairs):
        pairs = pairs + [(-1, -1)] * (2 - len(pairs))
        parents.copy_(i32([a for a, _ in pairs]))
        children.copy_(i32([b for _, b in pairs]))
        graphs[fork].replay()
        for a, b in pairs:
            if a >= 0:
                seqs[b] = list(seqs[a])

    def do_release(rows):
        e = [-(-len(seqs[n][0]) // s) if n in rows else 0 for n in range(N)]
        end.copy_(i32(e))
        graphs[release].replay()
        for n in rows:
            lens[n] = 0
            seqs[n] = [a[:0] for a in seqs[n]]

    append([29, 16, 0, 0, 0, 0])
    do_fork([(0, 2), (1, 3)])
    append([1, 3, 2, 9, 0, 0])
    do_fork([(2, 4), (0, 5)])
    append([5, 1, 1, 1, 11, 20])
    do_release([0, 3])
    graphs[compact].replay()
    used = {int(p) for n in range(N) for p in table[n, :-(-int(lens[n]) // s)]}
    assert used == set(range(len(used))) and state.tolist() == [0, P - len(used), 0]
    append([13, 2, 8, 0, 1, 7])
    do_fork([(4, 3)])
    append([1, 1, 1, 1, 1, 1])
    do_release(list(range(N)))
    assert state[1] == P and not holders.any()
    assert sorted(ring.tolist()) == list(range(P))


def test_pages_behind_a_window_are_released_early():
    """Entries wholly before the next token's window are let go, step by step; a fork afterwards shares only what
    is left, and the window's attention stays what it was."""
    s, width, P, W, D = 8, 16, 20, 20, 64
    z = lambda *n, dtype=torch.int32: torch.zeros(*n, dtype=dtype, device="cuda")
    lens, holders, state, ring = z(2), z(P), i32([0, P, 0]), i32(np.arange(P))
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    kc, vc = (torch.full((P, s, 1, D), float("nan"), device="cuda") for _ in range(2))
    seqs, rng = [[], []], np.random.default_rng(4)
    pages_ws = R.alloc_paged_pages_workspace(R.make_paged_shape(2, 0, num_pages=P, page_size=s, table_width=width))
    for m in ([50, 0], [9, 0], "fork", [3, 30], [10, 1]):
        if m == "fork":
            moves = z(1, 2)
            sh = R.make_paged_shape(2, 0, num_pages=P, page_size=s, table_width=width)
            R.paged_fork(sh, i32([0]), i32([1]), table, lens, holders, ring, state, table, lens, holders, moves, state)
            R.paged_copy(sh, moves, kc, vc)
            seqs[1] = list(seqs[0])
            continue
        T = sum(m)
        sh = R.make_paged_shape(2, T, 1, 1, D, P, s, width, io=torch.float32, window=W)
        q, k, v, o = (torch.from_numpy(rng.standard_normal((T, 1, D))).float().cuda() for _ in range(4))
        cu, pos, slots, lse = z(3), z(T), z(T, dtype=torch.int64), z(T, 1, dtype=torch.float32)
        R.paged_plan(sh, lens, i32(m), ring, state, table, cu, lens, pos, slots, state)
        assert state[2] == 0
        R.paged_kv_write(sh, k, v, slots, kc, vc)
        R.paged_attention(sh, q, kc, vc, table, cu, lens, 0.2, o, lse, R.alloc_paged_workspace(sh))
        R.paged_release(sh, z(2), ((lens - W + 1).clamp(min=0) // s).to(torch.int32), table, holders, ring, state, table, holders, state,
                        pages_ws)
        at = 0
        for n in range(2):
            if m[n]:
                seqs[n].append((f64(k)[at:at + m[n]], f64(v)[at:at + m[n]]))
                kf, vf = (np.concatenate([x[i] for x in seqs[n]])[None] for i in range(2))
                x = dict(q=q[at:at + m[n]], kc=torch.from_numpy(kf), vc=torch.from_numpy(vf), table=i32([[0]]),
                         cu=i32([0, m[n]]), kv=i32([kf.shape[1]]))
                compare(o[at:at + m[n]], lse[at:at + m[n]], expect(x, 0.2, W), "f32")
            at += m[n]
    held = {int(p) for p in table.flatten() if p >= 0}
    assert len(held) + int(state[1]) == P
