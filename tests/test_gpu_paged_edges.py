"""The paged cache at its edges: requests and row tiles without keys in the middle of a CTA's work, plans of
the largest sizes, and what a request's result may not depend on.  Tolerances as in test_gpu_paged.py."""
import os
import subprocess
import sys
import threading

import pytest
import torch

from linear_recurrent_rnn_gb300 import librglru as R
from test_gpu_paged import attend, build, compare, expect

pytestmark = pytest.mark.gpu


# (new, all) tokens of the requests, heads, window.  Every CTA has several items, among them runs of more
# items without keys than there are item records (4), after and before items with keys.
NO_KEYS = {
    "requests-without-keys": ([(1, 300), (1, 0), (1, 0), (1, 290), (1, 0)] * 26, 8, 8, 0),
    "a-request-without-keys-and-many-heads": (([(1, 200)] * 9 + [(1, 0)]) * 25, 16, 8, 0),
    "row-tiles-before-the-start": ([(1, 700)] * 160 + [(150, 9)] + [(1, 600)] * 160 + [(140, 0)] + [(1, 500)] * 50, 4, 2, 0),
    "row-tiles-before-the-start-window": ([(1, 900)] * 250 + [(150, 9)] + [(1, 800)] * 250 + [(140, 0)] + [(1, 700)] * 90,
                                          4, 2, 600),
    "only-items-without-keys": ([(1, 0)] * 200 + [(3, 0)], 4, 4, 0),
    "keys-last": ([(2, 0)] * 100 + [(1, 500)], 4, 4, 0),
}


@pytest.mark.parametrize("io,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64)])
@pytest.mark.parametrize("name", list(NO_KEYS))
def test_items_without_keys_among_others(name, io, D):
    lens, Hq, Hkv, window = NO_KEYS[name]
    x = build(lens, Hq, Hkv, D, 16, io, seed=len(lens) + D)
    o, L, ws = attend(x, D ** -0.5, window)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5, window), io)
    assert not ws[:256 + 4096].any()


@pytest.mark.parametrize("D", [64, 128, 256])
def test_row_tiles_without_keys_many_rows(D):
    """The same in the kernel for many rows a request: a chunk of many row tiles before position 0."""
    lens = [(60, 300), (3000, 40), (70, 70), (1500, 0), (60, 500)]
    x = build(lens, 4, 2, D, 16, "bf16", seed=D)
    o, L, ws = attend(x, D ** -0.5)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5), "bf16")


# ---------------------------------------------------------------- the plan's largest sizes
PLANS_IN_ORDER = """
import sys
sys.path[:0] = [{root!r}, {tests!r}]
import numpy as np
from oracle import paged as O
from test_gpu_paged import run_plan
for N in (4031, 4032, 4095, 4096):
    rng = np.random.default_rng(N)
    cached, new = rng.integers(0, 60, N), rng.integers(0, 2, N)
    table, free = rng.integers(0, 4 * N, (N, 4)), rng.permutation(4 * N)
    args = (cached, new, free, [3, N, 0], table, 16)
    for a, b in zip(run_plan(*args, 5000, False), O.plan(*args, 5000)):
        np.testing.assert_array_equal(a, b)
print("plans are right")
"""


def test_plans_about_the_default_shared_memory():
    """In a process of its own, from the smallest on: no larger call has raised the limit before."""
    tests = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", PLANS_IN_ORDER.format(root=os.path.dirname(tests), tests=tests)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "plans are right" in r.stdout, r.stdout + r.stderr


def test_plans_of_two_sizes_from_two_threads():
    """Each call takes the shared memory that it needs, whatever another thread calls for meanwhile."""
    i32 = dict(dtype=torch.int32, device="cuda")
    wrong = []

    def calls(N):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                sh = R.make_paged_shape(N, 1, num_pages=8, page_size=16, table_width=1)
                z = lambda n: torch.zeros(n, **i32)
                a = (z(N), z(N), z(8), z(3), z((N, 1)), z(N + 1), z(N), z(1), torch.zeros(1, dtype=torch.int64, device="cuda"), z(3))
                for _ in range(5000):
                    R.paged_plan(sh, *a)
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001  (reported by the test)
            wrong.append((N, e))

    threads = [threading.Thread(target=calls, args=(N,)) for N in (8192, 5000, 6000)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---------------------------------------------------------------- what a request's bits depend on
# (new, all) tokens: tiles of 16, 32 and 128 rows that are not full
UNSEEN = {"tiles-of-16": [(1, 300), (1, 77), (2, 131), (1, 20)], "tiles-of-32": [(5, 300), (4, 77), (6, 131), (5, 20)],
          "tiles-of-128": [(20, 300), (9, 77), (30, 131), (13, 20)]}


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(UNSEEN))
def test_unseen_values_change_no_bit(name, io):
    """Finite values, however large, in the other requests' queries, in padding rows and in cache
    slots past a request's length leave a request's output as it was, bit by bit."""
    lens = UNSEEN[name]
    x = build(lens, 8, 2, 64, 16, io, 21, spare_rows=6)
    T = sum(q for q, _ in lens)
    for c in ("kc", "vc"):
        x[c] = torch.nan_to_num(x[c], nan=0.0)
    x["q"][T:] = 0
    o, L, _ = attend(x, 0.125)
    g = torch.Generator(device="cuda").manual_seed(22)
    table = x["table"].cpu().numpy()
    for n, (_, kv) in enumerate(lens):
        if kv % 16:
            for c in ("kc", "vc"):
                stale = x[c][int(table[n, kv // 16]), kv % 16:]
                stale.copy_(torch.randn(stale.shape, generator=g, device="cuda") * 1000)
    x["q"][T:] = torch.randn(x["q"][T:].shape, generator=g, device="cuda").to(x["q"].dtype) * 1000
    o2, L2, _ = attend(x, 0.125)
    assert torch.equal(o, o2) and torch.equal(L, L2)
    for n in range(len(lens)):
        a, b = int(x["cu"][n]), int(x["cu"][n + 1])
        q = x["q"] * 300
        q[a:b] = x["q"][a:b]
        o2, L2, _ = attend(dict(x, q=q), 0.125)
        assert torch.equal(o[a:b], o2[a:b]) and torch.equal(L[a:b], L2[a:b])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 12, 40])
def test_scores_near_the_type_s_lowest(new, io):
    """Every score of a row far below -1e30, yet finite: with equal keys the weights are equal.  All
    values are 3, and so is every output."""
    x = build([(new, 64 + new)] * 2, 2, 1, 64, 16, io, 23)
    T, w = 2 * new, 64
    x["q"].fill_(-2.0 ** 58)
    x["kc"] = torch.where(torch.isnan(x["kc"]), x["kc"], torch.full_like(x["kc"], 2.0 ** 58))
    x["vc"] = torch.where(torch.isnan(x["vc"]), x["vc"], torch.full_like(x["vc"], 3.0))
    o, L, ws = attend(x, 1.0, w)
    assert R.rglru_sync_status(ws) == R.OK
    score = -64.0 * 2.0 ** 116
    assert score < -5e36
    assert (o == 3.0).all()
    assert ((L.double() / score - 1).abs() <= 2.0 ** -20).all()   # e of the module's tolerances, relative
