"""Further GPU tests of the cache in 4 bits (include/paged_q4.h).  Tolerances: those of test_gpu_paged_q4.py, which
says where they come from."""
import numpy as np
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


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("size", [20.0, 27.3, 29.55, 31.2])
@pytest.mark.parametrize("new", [1, 24])
def test_small_weights_with_few_and_many_rows(new, size, io):
    """One key with weight 1 and 120 000 with 2^-size each, whose values alone are not zero.  Weights enter as f16, held
    times 2^7 of the row's largest with many rows in bf16, else 2^11 (or as two numbers, 2^11): half of f16's smallest step,
    2^-25, is 2^-32 or 2^-36 of the largest for each key."""
    D, n = 64, 120001
    x = build([(new, n)], 1, 1, D, 16, io, 31, scales=(0x38, 0x39))  # scales 1
    x["q"].fill_(0.0)
    x["q"][..., 0] = 1.0
    page = int(x["table"][0, 0])
    for c in (x["cache"][0], x["cache"][2]):
        c.zero_()
    x["cache"][0][page, 0, 0, 0] = 0x07       # key 0: 6 in channel 0
    x["cache"][2][:] = 0x22                   # values 1, but key 0's 0
    x["cache"][2][page, 0] = 0
    scale = size * np.log(2.0) / 6            # scores size ln 2 and 0
    o, L, _ = attend(x, scale)
    *ref, _ = expect(x, scale)
    compare(o, L, (*ref, n * 2.0 ** (-32 if new > 16 and io == "bf16" else -36)), io)
    got = o[:, 0, 0].double().cpu().numpy()
    if size == 20.0:
        assert np.all(np.abs(got - (n - 1) * 2.0 ** -20 / (1 + (n - 1) * 2.0 ** -20)) < 1e-3)


# heads, head width, new tokens a request: tiles of 8 and 16 rows, and the kernel for many rows
LONG = {"8-rows": (2, 64, 1), "8-rows-128": (8, 128, 1), "8-rows-256": (4, 256, 1), "16-rows": (16, 64, 1), "16-rows-256": (10, 192, 1),
        "many-rows-64": (8, 64, 5), "many-rows-128": (16, 128, 4), "many-rows-256": (12, 256, 5)}


@pytest.mark.parametrize("name", list(LONG))
def test_float32_sums_over_long_contexts(name):
    """160 requests over one cache of 65536 keys, whose values are all 3: so is every output.  The tensor core cuts what it adds to a
    sum, to the sum's 24 bits; so float32 calls add up no more than 256 keys there (16 products of 16 keys), and those
    sums in float32.  Each of a product's 16 terms and the sum so far lose less than 2^-23 of that, half of it in the mean:
    17 / 2 * sum(k / 16, k <= 16) * 2^-23 = 72 * 2^-23 of the whole in the mean of all outputs, twice that in one.  Roundings
    to nearest, of 256 sums, 512 weights a thread and the weights' two f16 numbers, are no bias: at most
    (256 + 512) 2^-24 + 2^-22 in one output, 2^-22 in the mean of 160 and more rows."""
    Hq, D, new = LONG[name]
    n, N = 65536, 160
    x = build([(new, n)], Hq, 1, D, 16, "f32", 41)
    x["cache"][2].fill_(0x55)                 # 3
    c = x["cache"][3]
    c.copy_(torch.where(c == 0x7f, c, torch.full_like(c, 0x38)))
    _, _, _, Hkv, _, P, s, width = x["dims"]
    g = torch.Generator(device="cuda").manual_seed(1)
    x["q"] = torch.randn(N * new, Hq, D, generator=g, device="cuda")
    x["table"] = x["table"].repeat(N, 1).contiguous()
    x["cu"] = (torch.arange(N + 1, device="cuda") * new).to(torch.int32)
    x["kv"] = torch.full((N,), n, dtype=torch.int32, device="cuda")
    x["dims"] = (N, N * new, Hq, Hkv, D, P, s, width)
    o, _, ws = attend(x, 0.3 * D ** -0.5)
    assert R.rglru_sync_status(ws) == R.OK
    off = o.double() / 3 - 1
    assert abs(float(off.mean())) <= 72 * 2.0 ** -23 + 2.0 ** -22
    assert float(off.abs().max()) <= 144 * 2.0 ** -23 + 768 * 2.0 ** -24 + 2.0 ** -22
