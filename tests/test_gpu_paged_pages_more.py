"""Further GPU tests of the calls on a cache's pages (include/paged_pages.h), against their oracle: all equal."""
import numpy as np
import pytest

from oracle import paged_pages as O
from linear_recurrent_rnn_gb300 import librglru as R
from test_gpu_paged_pages import COMPACT_OUT, RELEASE_OUT, check, pool, run_compact, run_release

pytestmark = pytest.mark.gpu


def test_one_scratch_for_pools_of_any_size():
    """A scratch as large as the largest pool asks for serves all: what a call over a small pool leaves there would be
    pages to free, or in use, to a call over a larger one."""
    rng = np.random.default_rng(1)
    pools = [pool(rng, N, most, 16, spare, 0.3) for N, most, spare in ((4, 150, 30), (20, 900, 700), (60, 3000, 100000), (1, 30, 5), (9, 500, 4000))]
    largest = max(len(p[3]) for p in pools)
    ws = R.alloc_paged_pages_workspace(R.make_paged_shape(1, 0, num_pages=largest, page_size=16, table_width=1))
    for i in (0, 2, 1, 2, 4, 3, 2, 0, 4, 1):
        table, lens, holders, ring, state = pools[i]
        check(run_compact(lens, table, holders, ring, 16, i % 2 == 0, ws), O.compact(lens, table, holders, ring, 16), COMPACT_OUT)
        assert not ws.any()
        for j in (2, i):
            table, lens, holders, ring, state = pools[j]
            end = np.where(rng.random(len(lens)) < 0.6, -(-lens // 16), 0)
            want = O.release(lens * 0, end, table, holders, ring, state, table)
            check(run_release(lens * 0, end, table, holders, ring, state, True, ws), want, RELEASE_OUT)
            assert not ws.any()
