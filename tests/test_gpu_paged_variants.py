"""The attention over the paged cache across its kernels (chosen by the mean number of rows a
request, the width and the type), split items with many parts, non-finite neighbours, and a
device wait that runs out.  Tolerances as in test_gpu_paged.py."""
import numpy as np
import pytest
import torch

from linear_recurrent_rnn_gb300 import librglru as R
from oracle import paged as O
from test_gpu_paged import attend, build, compare, expect, f64, run_plan

pytestmark = pytest.mark.gpu

# (new, all) tokens of the requests, heads, head width, page, window
CASES = {
    "rows-20-64": ([(5, 90), (5, 5), (5, 300)], 8, 2, 64, 16, 0),
    "rows-20-128": ([(5, 130), (4, 4), (5, 261), (1, 1)], 8, 2, 128, 16, 0),
    "rows-20-256": ([(5, 130), (4, 150), (5, 261)], 8, 2, 256, 32, 70),
    "rows-32": ([(4, 129), (4, 640)], 8, 1, 128, 64, 0),
    "rows-16-of-16": ([(2, 400), (2, 77)], 8, 1, 128, 16, 0),
    "long-chunk-among-ones": ([(1, 200)] * 30 + [(41, 300), (1, 9)], 4, 2, 128, 16, 0),
    "long-chunk-among-ones-window": ([(1, 200)] * 30 + [(41, 300), (1, 9)], 4, 2, 64, 8, 50),
    "heads-32-of-one": ([(1, 300), (1, 33)], 32, 1, 128, 16, 0),
    "heads-48-of-one": ([(1, 300), (2, 33)], 48, 1, 64, 16, 0),
    "heads-7-of-one": ([(1, 300), (2, 33), (1, 130)], 14, 2, 192, 16, 0),
    "no-groups": ([(1, 100), (1, 513), (1, 1)], 3, 3, 256, 256, 0),
    "window-inside-a-page": ([(1, 1000), (3, 515)], 4, 4, 128, 256, 7),
    "one-request-many-parts": ([(1, 41000)], 4, 1, 64, 64, 0),
    "one-request-many-parts-32": ([(4, 30000)], 8, 1, 128, 16, 0),
    "one-chunk-many-parts": ([(70, 20000)], 2, 1, 64, 128, 0),
    "one-chunk-many-parts-256": ([(40, 9000)], 4, 1, 256, 16, 0),
}


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention_variants_match_oracle(name, io):
    lens, Hq, Hkv, D, s, window = CASES[name]
    x = build(lens, Hq, Hkv, D, s, io, seed=sum(map(ord, name)))
    o, L, ws = attend(x, D ** -0.5, window)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5, window), io)
    assert not ws[:256 + 4096].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_results_do_not_depend_on_the_batch(io):
    """A request alone and the same one among many, whose kernel, row tiles and parts differ."""
    lens = [(6, 700), (1, 300), (90, 400)]
    x = build(lens, 8, 2, 128, 16, io, 3)
    all_o, all_L, _ = attend(x, 0.09)
    for n, (q, kv) in enumerate(lens):
        a, b = int(x["cu"][n]), int(x["cu"][n + 1])
        dims = list(x["dims"])
        dims[0], dims[1] = 1, q
        y = dict(x, q=x["q"][a:b].contiguous(), table=x["table"][n:n + 1].contiguous(),
                 cu=torch.tensor([0, q], dtype=torch.int32, device="cuda"), kv=x["kv"][n:n + 1].contiguous(),
                 dims=tuple(dims))
        o, L, _ = attend(y, 0.09)
        ref = expect(y, 0.09)
        compare(o, L, ref, io)
        compare(all_o[a:b], all_L[a:b], ref, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_values_stay_with_their_request(new, bad, io):
    """A NaN or infinity in one request's keys, values or queries reaches no other request, and no
    token that does not see its position (decode steps and chunks; infinities give NaN through
    inf - inf, as the formula does)."""
    lens = [(new, 150), (new, 170), (new, 129)]
    x = build(lens, 4, 2, 64, 16, io, 4)
    ref = expect(x, 0.125)
    table = x["table"].cpu().numpy()
    x["kc"][table[1, 3], 5] = bad              # position 53 of request 1, seen by all its tokens
    x["vc"][table[1, 9], 2] = bad              # position 146
    x["q"][int(x["cu"][1])] = bad
    o, L, ws = attend(x, 0.125)
    assert R.rglru_sync_status(ws) == R.OK
    for n in (0, 2):
        a, b = int(x["cu"][n]), int(x["cu"][n + 1])
        compare(o[a:b], L[a:b], tuple(r[a:b] for r in ref), io)
    a, b = int(x["cu"][1]), int(x["cu"][2])
    assert not np.isfinite(f64(o[a:b])).any()


@pytest.mark.parametrize("rows", [1, 60])
def test_a_wait_that_runs_out_is_reported(rows):
    """One CTA hands its warps no work: their waits end after the given limit, the status says so,
    TMEM is free again, and after zeroing the workspace the next call is right."""
    x = build([(rows, 3000)], 4, 1, 128, 16, "bf16", 5)
    ws = attend(x, 0.1)[2]
    assert R.rglru_sync_status(ws) == R.OK
    R.rglru_debug_lookback(20000, 0)           # 2 ms
    try:
        attend(x, 0.1, ws=ws)
        assert R.rglru_sync_status(ws) == R.ERR_TIMEOUT
    finally:
        R.rglru_debug_lookback(0, -1)
    ws.zero_()
    o, L, _ = attend(x, 0.1, ws=ws)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, 0.1), "bf16")


def test_calls_launch_one_kernel_each():
    x = build([(3, 100), (1, 50)], 4, 2, 64, 16, "bf16", 6)
    before = R.rglru_kernel_launches()
    attend(x, 0.1)
    assert R.rglru_kernel_launches() == before + 1


def test_split_items_repeat_bitwise():
    """Items shared by two CTAs, either of which may finish last and join them, and row tiles with
    rows to spare (10 heads of one: 120 of 128): twenty runs give the same bits, whatever other
    calls left in the SMs' memory between them."""
    x = build([(1, 150), (173, 174), (173, 173), (1, 141), (173, 300)] * 6, 20, 2, 96, 16, "bf16", 9)
    other = build([(60, 190), (128, 1000)] * 20, 4, 4, 128, 16, "bf16", 10, k_scale=40.0)
    o, L, ws = attend(x, 96 ** -0.5)
    for _ in range(20):
        attend(other, 1.0)
        o2, L2, _ = attend(x, 96 ** -0.5, ws=ws)
        assert torch.equal(o, o2) and torch.equal(L, L2)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
@pytest.mark.parametrize("s", [8, 16, 32, 128])
def test_pages_and_widths(s, D, layout, new):
    """Pages from one swizzle atom to a whole tile, for widths with and without boxes of several
    column slabs: tiles cut at either end and inside a page, caches stored either way round."""
    lens = [(new, 300), (new, 131), (new, new), (new, 256)]
    for window in (0, 75):
        x = build(lens, 6, 2, D, s, "bf16", s + D, layout)
        o, L, ws = attend(x, D ** -0.5, window)
        assert R.rglru_sync_status(ws) == R.OK
        compare(o, L, expect(x, D ** -0.5, window), "bf16")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("N,tokens", [(1, 0), (1, 3), (32, 32), (33, 40), (513, 20), (513, 700), (1025, 1025), (2049, 5)])
def test_plan_where_its_warps_are_not_full(N, tokens, in_place):
    """Requests and rows about the sizes at which a warp, a CTA or a thread's share fills up; some
    requests past the table's width, rows short of the new tokens or beyond them."""
    rng = np.random.default_rng(N + tokens)
    cached = rng.integers(0, 60, N)
    new = np.where(rng.random(N) < min(1.0, tokens / N), rng.integers(0, 3, N), 0)
    P = 4 * N + 7
    table, free = rng.integers(0, P, (N, 4)), rng.permutation(P)
    args = (cached, new, free, [P - 3, N + 2, 0], table, 16)
    want = O.plan(*args, tokens)
    got = run_plan(*args, tokens, in_place)
    for n, a, b in zip(("table", "cu", "kv_lens", "positions", "slots", "state"), got, want):
        np.testing.assert_array_equal(a, b, err_msg=n)
