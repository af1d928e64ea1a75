"""Further GPU tests of the cache in 4 bits (include/paged_q4.h).  Tolerances: those of test_gpu_paged_q4.py, which
says where they come from."""
import pytest
import torch

from linear_recurrent_rnn_gb300 import librglru as R
from test_gpu_paged_q4 import attend, build, compare, expect

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (3, 1), (4, 1)])
@pytest.mark.parametrize("D", [144, 192, 256])
def test_wide_heads_with_up_to_four_rows(D, Hq, Hkv, window):
    """A step is two key tiles of four rows: half of what one read of the scores brings.  Keys that end before, at and
    behind a step's end, and requests that several CTAs share."""
    lens = [(1, n) for n in (1, 127, 128, 129, 255, 256, 257, 384, 511, 512, 513, 700, 5000)]
    x = build(lens, Hq, Hkv, D, 16, "bf16", seed=D + Hq)
    o, L, ws = attend(x, D ** -0.5, window)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5, window), "bf16")
