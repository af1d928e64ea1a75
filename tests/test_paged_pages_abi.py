"""CPU checks of the calls on a cache's pages (include/paged_pages.h): symbols, scratch, and refusals on the
host before any CUDA call (fake, never dereferenced addresses); and what its oracle leaves unchanged."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from linear_recurrent_rnn_gb300 import build as B_
from linear_recurrent_rnn_gb300 import librglru as R
from oracle import paged_pages as O
from test_paged_abi import A, BAD_CACHE, P, lib, shape  # noqa: F401  (lib: a fixture)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "paged_pages.h")
FORK = "parents children table lens holders ring state table_out lens_out holders_out moves out".split()
RELEASE = "first end table holders ring state table_out holders_out out ws".split()
COMPACT = "lens table holders table_out holders_out ring out moves ws".split()


def call(f, names, sh, head=(), **kw):
    a = dict({n: A for n in names}, **kw)
    return f(ctypes.byref(sh), *head, *[P(a[n]) for n in names], None)


def fork(lib, sh, n=2, **kw):  # noqa: F811
    return call(lib.paged_fork, FORK, sh, (n,), **kw)


def release(lib, sh, **kw):  # noqa: F811
    return call(lib.paged_release, RELEASE, sh, **kw)


def compact(lib, sh, **kw):  # noqa: F811
    return call(lib.paged_compact, COMPACT, sh, **kw)


def copy(lib, sh, n=2, moves=A, caches=(A,), strides=(64,), sizes=(64,), arrays=True):  # noqa: F811
    k = len(caches)
    ptr = (ctypes.c_void_p * max(k, 1))(*caches) if arrays else None
    i64 = lambda v: (ctypes.c_int64 * max(k, 1))(*v)
    return lib.paged_copy(ctypes.byref(sh), n, P(moves), k, ptr, i64(strides), i64(sizes), None)


def test_declared_symbols_are_exported(lib):  # noqa: F811
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(paged_[a-z_]+)\s*\(", src))
    assert names == set(R.EXPORTS_PAGES)
    out = subprocess.run(["nm", "-D", "--defined-only", B_.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (paged_\w+)", out))


@pytest.mark.parametrize("kw,want", BAD_CACHE + [(dict(num_seqs=8192, table_width=2 ** 18), R.ERR_UNSUPPORTED)])
def test_sizes_are_refused(lib, kw, want):  # noqa: F811
    for f in (fork, release, compact, copy):
        assert f(lib, shape(**kw)) == want
    assert R.paged_pages_workspace_bytes(shape(**kw)) == 0


def test_counts_are_refused(lib):  # noqa: F811
    assert fork(lib, shape(), -1) == R.ERR_INVALID_ARG
    assert fork(lib, shape(), 8193) == R.ERR_UNSUPPORTED
    assert copy(lib, shape(), -1) == R.ERR_INVALID_ARG


def test_pointers_are_refused(lib):  # noqa: F811
    for f, names in ((fork, FORK), (release, RELEASE), (compact, COMPACT)):
        for n in names:
            assert f(lib, shape(), **{n: None}) == R.ERR_INVALID_ARG, n
            assert f(lib, shape(), **{n: A + 2}) == R.ERR_INVALID_ARG, n
    assert copy(lib, shape(), moves=None) == R.ERR_INVALID_ARG
    assert copy(lib, shape(), moves=A + 2) == R.ERR_INVALID_ARG
    assert copy(lib, shape(), arrays=False) == R.ERR_INVALID_ARG
    assert copy(lib, shape(), caches=(None,)) == R.ERR_INVALID_ARG


def test_pages_that_overlap_or_are_too_long_are_refused(lib):  # noqa: F811
    for stride, size, want in ((64, 0, R.ERR_INVALID_ARG), (63, 64, R.ERR_INVALID_ARG), (-64, 64, R.ERR_INVALID_ARG),
                               (1 << 30, (1 << 28) + 1, R.ERR_UNSUPPORTED)):
        assert copy(lib, shape(), caches=(A, A), strides=(64, stride), sizes=(64, size)) == want


def test_no_moves_are_no_work(lib):  # noqa: F811
    assert copy(lib, shape(), 0, moves=None) == R.OK
    assert copy(lib, shape(), 2, caches=(), strides=(), sizes=(), arrays=False) == R.OK


def test_the_binding_refuses_wrong_tensors(lib):  # noqa: F811
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="^parents: "):   # not on a GPU
        R.paged_fork(shape(), z, z, z, z, z, z, z, z, z, z, z, z)
    with pytest.raises(ValueError, match="^first_pages: "):
        R.paged_release(shape(), z, z, z, z, z, z, z, z, z, z)
    with pytest.raises(TypeError, match="^kv_lens: "):
        R.paged_compact(shape(), 3, z, z, z, z, z, z, z, z)
    with pytest.raises(ValueError, match="^moves: "):
        R.paged_copy(shape(), z, z)


# ---------------------------------------------------------------- the oracle
def pool(seed, N=6, width=7, P=40, s=16):
    """Rows of random lengths over a pool: (table, lens, holders, ring, state)."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, width * s + 1, N)
    held = -(-lens // s)
    ids = rng.permutation(max(P, int(held.sum()) + 9))
    P = len(ids)
    table = np.full((N, width), -1, np.int64)
    at = 0
    for n in range(N):
        table[n, :held[n]] = ids[at:at + held[n]]
        at += held[n]
    ring, head = np.full(P, -1, np.int64), int(rng.integers(0, P))
    ring[(head + np.arange(P - at)) % P] = ids[at:]
    return table, lens, np.zeros(P, np.int64), ring, [head, P - at, 0]


def in_ring(ring, state):
    return [int(ring[(state[0] + i) % len(ring)]) for i in range(state[1])]


@pytest.mark.parametrize("seed", range(4))
def test_oracle_fork_then_release_gives_every_page_back(seed):
    """After a fork the children's tokens are where the parents' are, or in pages to be copied; with all rows
    released every page is on the ring once."""
    table, lens, holders, ring, state = pool(seed)
    N, width = table.shape
    big = np.vstack([table, np.full((3, width), -1)])
    all_lens = np.concatenate([lens, [0, 0, 0]])
    out, L, held, moves, st = O.fork([1, 1, 4], [8, 6, 7], big, all_lens, holders, ring, state, 16, big, all_lens)
    assert list(L[6:]) == [lens[1], lens[4], lens[1]]
    data = np.random.default_rng(seed).standard_normal((len(ring), 16))
    data2 = O.copy(data, moves)
    for c, p in ((8, 1), (6, 1), (7, 4)):
        for t in range(lens[p]):
            assert data2[out[c, t // 16], t % 16] == data[table[p, t // 16], t % 16]
    end = -(-L // 16)
    t3, h3, r3, s3 = O.release(np.zeros(N + 3, int), end, out, held, ring, st, out)
    assert (t3 == -1).all() and (h3 == 0).all() and s3[1] == len(ring)
    assert sorted(in_ring(r3, s3)) == list(range(len(ring)))


@pytest.mark.parametrize("seed", range(4))
def test_oracle_compact_keeps_what_the_rows_hold(seed):
    table, lens, holders, ring, state = pool(seed)
    holders = np.random.default_rng(seed).integers(0, 3, len(holders))
    out, held, r, st, moves = O.compact(lens, table, holders, ring, 16)
    data = np.random.default_rng(seed).standard_normal((len(ring), 16))
    data2 = O.copy(data, moves)
    U = len(ring) - st[1]
    for n, L in enumerate(lens):
        for t in range(L):
            assert out[n, t // 16] < U and data2[out[n, t // 16], t % 16] == data[table[n, t // 16], t % 16]
            assert held[out[n, t // 16]] == holders[table[n, t // 16]]
    assert sorted(in_ring(r, st)) == list(range(U, len(ring)))
