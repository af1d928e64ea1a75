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


@pytest.mark.parametrize("io,Hq,D", [("bf16", 4, 64), ("bf16", 8, 128), ("bf16", 4, 256), ("bf16", 7, 192), ("f32", 5, 128), ("f32", 8, 256)])
def test_items_of_one_step_give_the_same_bits_every_time(io, Hq, D):
    """The references move in an item's only step; its sums follow at once.  More items a CTA than it has records, rows
    of different sizes."""
    x = build([(1, 1 + n * 37 % (2 * 128)) for n in range(1500)], Hq, 1, D, 16, io, seed=D)
    x["q"] *= torch.exp2(torch.arange(Hq, device="cuda") % 4).to(x["q"].dtype)[:, None]
    o, L, ws = attend(x, D ** -0.5)
    compare(o, L, expect(x, D ** -0.5), io)
    for _ in range(30):
        o2, L2, _ = attend(x, D ** -0.5, ws=ws)
        assert torch.equal(o, o2) and torch.equal(L, L2)
