"""The paged cache at its edges: requests and row tiles without keys in the middle of a CTA's work.
Tolerances as in test_gpu_paged.py."""
import pytest

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
