"""GPU parity of the cache in 4 bits (include/paged_q4.h) with its oracle: the write code by code, the read
exactly, the attention element by element against oracle.paged over the values that the cache stands for.

Tolerances of the attention, from its arithmetic.  With A = sum_j p_j |v_j|, B = max_j sum_d |scale q_d k_jd|, n keys:
  keys and values enter exactly.  Queries: bf16 exactly (f16 has 11 bits; elements of a row below 2^-29 of its largest
  lose bits, at most 2^-39 of the largest); float32 as two f16 numbers, 2^-22 of an element, or 2^-39 of the row's
  largest where that is more.  Sums of D products: 2^-20 B (as for the other cache), the exponent's argument and
  function 2^-21.  So lse is off by at most e = (2^-20 + 2^-22 [float32]) B + 2^-39 scale max|q| max_j sum_d |k_jd| +
  2^-21 max(1, |lse|).
  Weights: f16, 2^-11 (half its spacing), or two f16 numbers, 2^-22; a weight is held times 2^11 of the largest, so what
  f16's smallest step, 2^-24, rounds away is at most 2^-36 of the largest each.  So o is off by at most
  (2 e + 2^-20 + 2^-11 or 2^-22) A + n 2^-36 max|v|, and half a bf16 spacing for its own rounding."""
import numpy as np
import pytest
import torch

from helpers import half_ulp_bf16
from oracle import paged as P_
from oracle import paged_q4 as O
from linear_recurrent_rnn_gb300 import librglru as R
from test_gpu_paged import DT, f64

pytestmark = pytest.mark.gpu

E4 = torch.float8_e4m3fn


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == E4 else t.cpu().numpy()


def layout(P, s, H, width, pad, kind):
    """A [P, s, H, width] view of bytes: head by head (as alloc_paged_q4_cache), token by token, or a part of a larger block."""
    w = -(-width // pad) * pad
    if kind == "hnd":
        return torch.zeros(P, H, s, w, dtype=torch.uint8, device="cuda")[..., :width].transpose(1, 2)
    if kind == "nhd":
        return torch.zeros(P, s, H, w, dtype=torch.uint8, device="cuda")[..., :width]
    return torch.zeros(P, 3, s, H, w, dtype=torch.uint8, device="cuda")[:, 1, ..., :width]


def new_cache(P, s, H, D, kind="hnd"):
    return [layout(P, s, H, D // 2, 16, kind), layout(P, s, H, D // 16, 4, kind),
            layout(P, s, H, D // 2, 16, kind), layout(P, s, H, D // 16, 4, kind)]


def as_scales(cache):
    return [c.view(E4) if i % 2 else c for i, c in enumerate(cache)]


# ---------------------------------------------------------------- write and read
def groups(io, rng, n):
    """n groups of 16: ordinary ones of many sizes, and those where a border between codes or scales is met."""
    dt = DT[io]
    x = torch.from_numpy(rng.standard_normal((n, 16)) * np.exp(rng.standard_normal((n, 1)) * 3)).to(dt)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.25, -0.75, -1.75, -5.0, 4.0, -0.0, 0.5])
    for i in range(n // 4):  # borders exactly, and the numbers next to them
        s = float(O.E4M3[rng.integers(1, 127)])
        y = (mids * s).to(dt)
        if i % 3:
            step = torch.from_numpy(rng.integers(-1, 2, 16)).to(torch.int16 if io == "bf16" else torch.int32)
            step[[7, 8, 14]] = 0  # (the largest stays, and the zeros)
            y = (y.view(step.dtype) + step).view(dt)
        x[i] = y
    for i in range(n // 4, n // 2):  # largest elements at and next to a border between scales
        c = int(rng.integers(0, 126))
        a = torch.tensor([6 * (O.E4M3[c] + O.E4M3[c + 1]) / 2]).to(dt)
        k = torch.int16 if io == "bf16" else torch.int32
        a = (a.view(k) + int(rng.integers(-1, 2))).view(dt)
        x[i] = (torch.from_numpy(rng.uniform(-1, 1, 16)) * float(a)).to(dt)
        x[i, rng.integers(16)] = float(a)
    big = torch.finfo(dt).max
    for i, v in enumerate([0.0, -0.0, float("nan"), float("inf"), -float("inf"), big, 2688.0, 2700.0, 5000.0, 1e-30, 2.0 ** -126,
                           2.0 ** -133, 6 * 2.0 ** -10, 6 * 2.0 ** -9, 3e38]):
        x[-1 - i] = torch.from_numpy(rng.uniform(-1, 1, 16)).to(dt) if abs(v) < 1e4 and v != 0 else 0.0
        if v == v and abs(v) < 1e5:
            x[-1 - i] *= v
        x[-1 - i, i] = v
    return x


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_codes_and_scales_are_the_nearest(io):
    rng = np.random.default_rng(1)
    H, D, s, T = 2, 64, 16, 100
    x = groups(io, rng, 2 * T * H * D // 16).view(2, T, H, D)
    k, v = x[0].cuda(), x[1].cuda()
    cache = new_cache(8, s, H, D)
    slots = torch.from_numpy(rng.permutation(8 * s)[:T]).cuda()
    sh = R.make_paged_shape(1, T, H, H, D, 8, s, 1, io=DT[io])
    R.paged_q4_write(sh, k, v, slots, *as_scales(cache))
    at = slots.cpu().numpy()
    for i, src in enumerate((x[0], x[1])):
        want = O.quantise(src.double().numpy())
        for got, w in zip(cache[2 * i:2 * i + 2], want):
            np.testing.assert_array_equal(got.cpu().numpy()[at // s, at % s], w)
    # and read back: what the codes stand for, exactly
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    R.paged_q4_read(sh, slots, *as_scales(cache), ko, vo)
    for i, got in enumerate((ko, vo)):
        np.testing.assert_array_equal(f64(got), O.values(*O.quantise(x[i].double().numpy())))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,s,kind", [(1, 1, 16, 8, "hnd"), (7, 3, 80, 16, "hnd"), (9, 1, 48, 8, "nhd"), (65, 1, 256, 32, "block"),
                                          (33, 2, 96, 64, "nhd"), (5, 9, 128, 16, "hnd"), (3, 1, 240, 8, "hnd")])
def test_write_touches_its_slots_alone(T, H, D, s, kind, io):
    """Every other byte of the caches, paddings and neighbours among them, keeps its value."""
    rng = np.random.default_rng(T + D)
    P = -(-T // s) + 2
    cache = new_cache(P, s, H, D, kind)
    whole = [c._base for c in cache]
    for b in whole:
        b.copy_(torch.from_numpy(rng.integers(0, 256, tuple(b.shape)).astype(np.uint8)))
    before = [c.cpu().numpy() for c in cache]
    held = [b.clone() for b in whole]
    kv = torch.from_numpy(rng.standard_normal((T, 2 * H, D))).to(DT[io]).cuda()
    slots = rng.permutation(P * s)[:T].astype(np.int64)
    if T > 5:
        slots[[1, 3, 5]] = [-1, P * s, 2 ** 40]
    sh = R.make_paged_shape(1, T, H, H, D, P, s, 1, io=DT[io])
    R.paged_q4_write(sh, kv[:, :H], kv[:, H:], torch.from_numpy(slots).cuda(), *as_scales(cache))
    for i, part in enumerate((kv[:, :H], kv[:, H:])):
        for c, w, b in zip(cache[2 * i:2 * i + 2], O.quantise(f64(part)), before[2 * i:2 * i + 2]):
            np.testing.assert_array_equal(c.cpu().numpy(), P_.write(b, w, slots))
    for c, v, b, h in zip(cache, before, whole, held):
        c.copy_(torch.from_numpy(v))
        assert torch.equal(b, h)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_read_of_any_bytes(io):
    """All codes and scales, negative and NaN ones among them; slots that repeat, and slots outside."""
    rng = np.random.default_rng(2)
    P, s, H, D = 4, 16, 3, 96
    cache = new_cache(P, s, H, D)
    for c in cache:
        c.copy_(torch.from_numpy(rng.integers(0, 256, tuple(c.shape)).astype(np.uint8)))
    slots = rng.integers(0, P * s, 50).astype(np.int64)
    slots[[0, 9, 49]] = [-1, P * s, -2 ** 40]
    sh = R.make_paged_shape(1, 50, H, H, D, P, s, 1, io=DT[io])
    wide = [torch.full((50, 5, D), 7.0, dtype=DT[io], device="cuda") for _ in range(2)]
    R.paged_q4_read(sh, torch.from_numpy(slots).cuda(), *as_scales(cache), *(w[:, 1:4] for w in wide))
    there = (slots >= 0) & (slots < P * s)
    at = np.where(there, slots, 0)
    for i, w in enumerate(wide):
        want = O.values(*(c.cpu().numpy()[at // s, at % s] for c in cache[2 * i:2 * i + 2]))
        want[~there] = 0.0
        np.testing.assert_array_equal(f64(w[:, 1:4]), want)
        assert (w[:, 0] == 7).all() and (w[:, 4] == 7).all()


# ---------------------------------------------------------------- attention
def build(lens, Hq, Hkv, D, s, io, seed, kind="hnd", fused=False, spare_rows=0, scales=(0x18, 0x2c)):
    """Requests of (new, all) tokens in scattered pages of a cache that is NaN wherever no request has a token, with
    garbage in the table past each request's pages.  Random codes; scales drawn from a range of E4M3 codes."""
    rng = np.random.default_rng(seed)
    N = len(lens)
    used = [-(-kv // s) for _, kv in lens]
    P = sum(used) + 3
    width = max(used + [1]) + 2
    ids = rng.permutation(P)
    table = rng.choice([-1, 0, P - 1, P, 2 ** 30], size=(N, width)).astype(np.int32)
    cache = new_cache(P, s, Hkv, D, kind)
    host = [np.zeros(tuple(c.shape), np.uint8) for c in cache]
    for i in (0, 2):
        host[i][:] = rng.integers(0, 256, host[i].shape)
        host[i + 1][:] = 0x7f
    at = 0
    for n, (_, kv) in enumerate(lens):
        table[n, :used[n]] = ids[at:at + used[n]]
        at += used[n]
        j = np.arange(kv)
        pg = table[n, j // s] if kv else j
        for i in (1, 3):
            host[i][pg, j % s] = rng.integers(*scales, (kv,) + host[i].shape[2:])
    for c, h in zip(cache, host):
        c.copy_(torch.from_numpy(h))
    T = sum(q for q, _ in lens) + spare_rows
    qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, D))).to(DT[io]).cuda()
    q = qkv[:, :Hq] if fused else qkv[:, :Hq].contiguous()
    cu = np.concatenate([[0], np.cumsum([q_ for q_, _ in lens])]).astype(np.int32)
    return dict(q=q, cache=cache, table=torch.from_numpy(table).cuda(), cu=torch.from_numpy(cu).cuda(),
                kv=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
                dims=(N, T, Hq, Hkv, D, P, s, width), io=io)


def attend(x, scale, window=0, ws=None, o=None, lse=True, stream=None):
    sh = R.make_paged_shape(*x["dims"], io=DT[x["io"]], window=window)
    ws = R.alloc_paged_q4_workspace(sh) if ws is None else ws
    T, Hq, D = x["q"].shape
    o = torch.full((T, Hq, D), 77.0, dtype=x["q"].dtype, device="cuda") if o is None else o
    L = torch.full((T, Hq), 77.0, device="cuda") if lse else None
    R.paged_q4_attention(sh, x["q"], *as_scales(x["cache"]), x["table"], x["cu"], x["kv"], scale, o, L, ws, stream)
    return o, L, ws


def expect(x, scale, window=0):
    kc, vc = (O.values(*(c.cpu().numpy() for c in x["cache"][i:i + 2])) for i in (0, 2))
    ref = P_.attention(f64(x["q"]), kc, vc, x["table"].cpu().numpy(), x["cu"].cpu().numpy(), x["kv"].cpu().numpy(), scale, window)
    biggest = lambda c: float(np.nanmax(np.abs(c), initial=0.0))
    with np.errstate(invalid="ignore"):
        floor = 2.0 ** -39 * scale * biggest(f64(x["q"])) * float(np.nanmax(np.abs(kc).sum(-1), initial=0.0))
    return ref + (floor, int(x["kv"].max()) * 2.0 ** -36 * biggest(vc))


def compare(o, L, ref, io):
    ro, rl, av, qk, floor, lost = ref
    live = ~np.isnan(rl)
    o = f64(o)
    assert np.all(o[~live] == 77.0)
    f32 = io == "f32"
    e = (2.0 ** -20 + 2.0 ** -22 * f32) * qk + floor + 2.0 ** -21 * np.maximum(1.0, np.abs(np.where(np.isfinite(rl), rl, 0.0)))
    tol = (2 * e[..., None] + 2.0 ** -20 + (2.0 ** -22 if f32 else 2.0 ** -11)) * av + lost
    if not f32:
        tol = tol + half_ulp_bf16(np.abs(ro) + tol)
    d = np.abs(o[live] - ro[live])
    assert np.all(np.isfinite(o[live]))
    worst = np.max(d / np.maximum(tol[live], 1e-30)) if d.size else 0.0
    assert np.all(d <= tol[live]), f"o: {worst:.2f} of the tolerance, max {d.max():.3e}"
    if L is not None:
        L = f64(L)
        assert np.all(L[~live] == 77.0)
        none = live & (rl == -np.inf)
        assert np.all(L[none] == -np.inf) and np.all(o[none] == 0.0)
        some = live & np.isfinite(rl)
        dl = np.abs(L[some] - rl[some])
        assert np.all(dl <= e[some]), f"lse: {np.max(dl / e[some]):.2f} of the tolerance"


# (new, all) tokens of the requests, heads, head width, page, window
CASES = {
    "one-token": ([(1, 1)], 1, 1, 64, 16, 0),
    "decode": ([(1, 1), (1, 2), (1, 127), (1, 128), (1, 129), (1, 600)], 8, 2, 128, 16, 0),
    "decode-mqa-256": ([(1, 300), (1, 17), (1, 1000)], 10, 1, 256, 32, 0),
    "decode-window": ([(1, 700), (1, 64), (1, 65), (1, 3)], 4, 4, 64, 64, 64),
    "drafts": ([(5, 130), (4, 4), (7, 261), (1, 1)], 16, 2, 128, 8, 0),
    "prefill": ([(200, 200), (129, 129), (1, 1), (64, 64)], 4, 2, 64, 16, 0),
    "prefill-long": ([(700, 700)], 2, 1, 128, 128, 0),
    "chunks": ([(33, 400), (128, 257), (100, 1111)], 6, 2, 128, 64, 0),
    "chunks-window": ([(300, 900), (50, 51), (129, 640)], 4, 1, 128, 16, 100),
    "window-one": ([(40, 90), (3, 3)], 2, 2, 64, 16, 1),
    "empty-requests": ([(0, 50), (3, 20), (0, 0), (2, 300), (0, 7)], 4, 4, 64, 16, 0),
    "rows-before-the-start": ([(5, 2), (4, 0), (1, 0), (200, 90)], 4, 2, 64, 16, 0),
    "width-80": ([(9, 140), (130, 131)], 3, 3, 80, 32, 0),
    "width-16": ([(3, 30)], 2, 1, 16, 8, 0),
    "width-48": ([(3, 130), (1, 9)], 2, 2, 48, 8, 0),
    "width-208": ([(5, 150), (70, 70)], 5, 1, 208, 16, 33),
    "prefill-256": ([(150, 150), (90, 300)], 4, 2, 256, 64, 0),
    "width-192": ([(1, 150), (9, 300)], 4, 2, 192, 8, 0),
    "group-5": ([(40, 200), (1, 77)], 10, 2, 96, 16, 0),
    "group-64": ([(3, 140), (1, 500)], 64, 1, 128, 16, 0),
    "group-33": ([(1, 140), (2, 300)], 66, 2, 64, 16, 0),
    "group-17-long": ([(60, 200), (2, 300)], 17, 1, 256, 16, 40),
    "group-12": ([(1, 500), (1, 33), (1, 1)], 12, 1, 128, 16, 0),
    "group-12-64": ([(1, 500), (1, 129)], 24, 2, 64, 32, 200),
    "group-20-256": ([(1, 300), (1, 40)], 20, 1, 256, 16, 0),
    "group-40-192": ([(1, 700), (0, 9), (1, 127)], 40, 1, 192, 8, 0),
    "prompts-64": ([(300, 300), (290, 500)], 16, 2, 64, 16, 0),
    "prompts-80": ([(200, 450)], 8, 1, 80, 16, 130),
    "prompts-128": ([(260, 700), (300, 300), (250, 900)], 10, 2, 128, 32, 0),
    "page-4096": ([(3, 5000)], 2, 1, 64, 4096, 0),
    "mixed": ([(1, 350)] * 6 + [(160, 320), (1, 1), (77, 900)], 8, 1, 128, 16, 256),
}


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_attention_matches_oracle(name, io):
    lens, Hq, Hkv, D, s, window = CASES[name]
    x = build(lens, Hq, Hkv, D, s, io, seed=sum(map(ord, name)))
    o, L, ws = attend(x, D ** -0.5, window)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5, window), io)
    assert not ws[:256 + 4096].any()   # counters as they were: zero


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["nhd", "block"])
@pytest.mark.parametrize("D", [64, 80])
def test_attention_strided(kind, D, io):
    """Caches stored token by token or as a part of a larger block, queries as slices of a fused projection, the
    output inside a wider buffer, padding rows, no lse."""
    x = build([(20, 150), (1, 40), (3, 3)], 6, 2, D, 16, io, 5, kind, fused=True, spare_rows=4)
    T = x["q"].shape[0]
    wide = torch.full((T, 9, D), 77.0, dtype=DT[io], device="cuda")
    o, _, _ = attend(x, 0.2, o=wide[:, 2:8], lse=False)
    assert torch.all(wide[:, :2] == 77.0) and torch.all(wide[:, 8:] == 77.0)
    compare(o, None, expect(x, 0.2), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(140, 700), (1, 400)], [(1, 700), (2, 400)]])
def test_attention_large_scores(lens, io):
    """Scores of some hundreds: the running maximum moves far, weights underflow."""
    x = build(lens, 2, 1, 128, 16, io, 6, scales=(0x30, 0x50))
    o, L, _ = attend(x, 128 ** -0.5)
    compare(o, L, expect(x, 128 ** -0.5), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-36, 1e-20, 1e15, 1e30])
def test_queries_of_any_size(size, io):
    """A row's size changes with its row; f16 could hold none of them."""
    x = build([(3, 200), (1, 90)], 4, 2, 64, 16, io, 8)
    grow = torch.tensor([1.0, 2.0 ** -40, 2.0 ** 9, 0.0], device="cuda")[:, None]
    x["q"] = (x["q"].double() * grow * size).to(DT[io])
    scale = 1.0 / (64 * size)
    o, L, _ = attend(x, scale)
    compare(o, L, expect(x, scale), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(3, 400), (1, 290)], [(300, 900)]])
def test_scales_that_leave_nothing_of_the_scores(lens, io):
    """Queries of zero (and tiny ones) with a tiny scale: every key that a row sees weighs the same, behind tiles
    of which it sees nothing (the rows of a tile see windows that begin in several of them)."""
    x = build(lens, 4, 2, 64, 16, io, 9)
    x["q"][:, 0] = 0
    x["q"][:, 1:] *= 1e-30
    for scale in (1e-12, 1e-37):
        o, L, _ = attend(x, scale, 70)
        compare(o, L, expect(x, scale, 70), io)


@pytest.mark.parametrize("Hq,D,io", [(4, 64, "bf16"), (24, 64, "bf16"), (10, 256, "f32"), (48, 256, "f32")])
def test_as_many_requests_as_there_may_be(Hq, D, io):
    """8192 of them, most without a token; few and many rows a request."""
    x = build([(1, 1 + n % 45) if n % 28 == 0 else (0, n % 3 * 7) for n in range(8192)], Hq, 1, D, 16, io, 31)
    o, L, ws = attend(x, D ** -0.5)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_repeats_bitwise_and_keeps_its_workspace(io):
    """Many CTAs share a request's keys: a second run on the same workspace, and one on another stream with its
    own, give the same bits."""
    x = build([(1, 9000), (3, 4000)], 4, 1, 128, 16, io, 7)
    o1, L1, ws = attend(x, 0.1)
    o2, L2, _ = attend(x, 0.1, ws=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o3, L3, _ = attend(x, 0.1)
    torch.cuda.synchronize()
    for o, L in ((o2, L2), (o3, L3)):
        assert torch.equal(o, o1) and torch.equal(L, L1)
    compare(o1, L1, expect(x, 0.1), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_table_entries_outside_the_cache_read_as_zeros(io):
    x = build([(2, 60), (1, 40)], 2, 1, 64, 16, io, 8)
    x["table"][0, 1] = -7
    x["table"][1, 0] = x["dims"][5]
    x["kv"][1] = 16 * x["dims"][7] + 5
    x["table"][1, 1:] = x["table"][0, 0]   # a whole page: all finite
    o, L, _ = attend(x, 0.2)
    compare(o, L, expect(x, 0.2), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_offsets_out_of_range_stay_in_bounds(io):
    x = build([(3, 20), (2, 30)], 2, 1, 64, 16, io, 9)
    for cu in ([0, 3, 900], [4, 2, -5], [-3, 2 ** 31 - 1, 1]):
        x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        x["kv"] = torch.tensor([20, -4], dtype=torch.int32, device="cuda")
        buf = torch.full((5 + 64, 2, 64), 77.0, dtype=DT[io], device="cuda")
        _, _, ws = attend(x, 0.2, o=buf[32:37])
        assert R.rglru_sync_status(ws) == R.OK
        assert torch.all(buf[:32] == 77.0) and torch.all(buf[37:] == 77.0)


# Runs of more items without keys than there are item records (4), after and before items with keys.
NO_KEYS = {
    "requests-without-keys": ([(1, 300), (1, 0), (1, 0), (1, 290), (1, 0)] * 26, 8, 8, 0),
    "row-tiles-before-the-start": ([(1, 700)] * 160 + [(150, 9)] + [(1, 600)] * 160 + [(140, 0)] + [(1, 500)] * 50, 4, 2, 0),
    "row-tiles-before-the-start-window": ([(1, 900)] * 250 + [(150, 9)] + [(1, 800)] * 250 + [(140, 0)] + [(1, 700)] * 90, 4, 2, 600),
    "only-items-without-keys": ([(1, 0)] * 200 + [(3, 0)], 4, 4, 0),
    "keys-last": ([(2, 0)] * 100 + [(1, 500)], 4, 4, 0),
}


@pytest.mark.parametrize("io,D", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("f32", 64), ("f32", 256)])
@pytest.mark.parametrize("name", list(NO_KEYS))
def test_items_without_keys_among_others(name, io, D):
    lens, Hq, Hkv, window = NO_KEYS[name]
    x = build(lens, Hq, Hkv, D, 16, io, seed=len(lens) + D)
    o, L, ws = attend(x, D ** -0.5, window)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, D ** -0.5, window), io)
    assert not ws[:256 + 4096].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[(1, 300), (1, 77), (2, 131), (1, 20)], [(5, 300), (4, 77), (6, 131), (5, 20)],
                                  [(20, 300), (9, 77), (30, 131), (13, 20)]])
def test_unseen_values_change_no_bit(lens, io):
    """The other requests' queries, padding rows and cache slots past a request's length leave a request's output as
    it was, bit by bit, NaN and infinities among them."""
    x = build(lens, 8, 2, 64, 16, io, 21, spare_rows=6)
    T = sum(q for q, _ in lens)
    o, L, _ = attend(x, 0.125)
    table = x["table"].cpu().numpy()
    for n, (_, kv) in enumerate(lens):
        if kv % 16:
            for i in (1, 3):
                x["cache"][i][int(table[n, kv // 16]), kv % 16:] = 0x7e
    x["q"][T:] = float("nan")
    o2, L2, _ = attend(x, 0.125)
    assert torch.equal(o[:T], o2[:T]) and torch.equal(L[:T], L2[:T])
    for n in range(len(lens)):
        a, b = int(x["cu"][n]), int(x["cu"][n + 1])
        q = torch.full_like(x["q"], float("inf")) if n % 2 else x["q"] * 300
        q[a:b] = x["q"][a:b]
        o2, L2, _ = attend(dict(x, q=q), 0.125)
        assert torch.equal(o[a:b], o2[a:b]) and torch.equal(L[a:b], L2[a:b])


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 12, 40])
def test_scores_near_the_type_s_lowest(new, io):
    """Every score of a row far below -1e30, yet finite: with equal keys the weights are equal.  All values are 3,
    and so is every output."""
    x = build([(new, 64 + new)] * 2, 2, 1, 64, 16, io, 23)
    x["q"].fill_(-2.0 ** 100)
    for i, (code, scale) in enumerate([(0x66, 0x78), (0x22, 0x44)]):  # 4 x 256 = 2^10; 1 x 3
        x["cache"][2 * i].fill_(code)
        c = x["cache"][2 * i + 1]
        c.copy_(torch.where(c == 0x7f, c, torch.full_like(c, scale)))
    o, L, ws = attend(x, 2.0 ** 6, 64)
    assert R.rglru_sync_status(ws) == R.OK
    score = -64.0 * 2.0 ** 116
    assert (o == 3.0).all()
    assert ((L.double() / score - 1).abs() <= 2.0 ** -20).all()


def test_many_small_weights_count():
    """One key with weight 1 and 120 000 with 2^-20 each, whose values alone are not zero: their sum is an eighth of the
    output's denominator, and f16 could not hold such weights beside 1 unscaled."""
    D, n = 64, 120001
    for io in ("bf16", "f32"):
        x = build([(1, n)], 1, 1, D, 16, io, 31, scales=(0x38, 0x39))  # scales 1
        x["q"].fill_(0.0)
        x["q"][..., 0] = 1.0
        table = x["table"].cpu().numpy()
        for c in (x["cache"][0], x["cache"][2]):
            c.zero_()
        page, off = int(table[0, 0]), 0
        x["cache"][0][page, off, 0, 0] = 0x07     # key 0: 6 in channel 0
        x["cache"][2][:] = 0x22                   # values 1, but key 0's 0
        x["cache"][2][page, off] = 0
        x["cache"][1][page, off] = 0x38
        scale = 20 * np.log(2.0) / 6              # scores 20 ln 2 and 0
        o, L, _ = attend(x, scale)
        compare(o, L, expect(x, scale), io)
        assert abs(float(o[0, 0, 0]) - (n - 1) * 2.0 ** -20 / (1 + (n - 1) * 2.0 ** -20)) < 1e-3


def test_a_long_cache_whose_offsets_pass_32_bits():
    P, s, H, D = 17000, 4096, 2, 128
    sh = R.make_paged_shape(1, 5, H, H, D, P, s, 1, io=R.BF16, window=5)
    cache = R.alloc_paged_q4_cache(sh)
    assert cache[0].numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    q, k, v = (torch.randn(5, H, D, generator=g, device="cuda").bfloat16() for _ in range(3))
    slots = (P - 1) * s + torch.arange(5, device="cuda") + 4000
    R.paged_q4_write(sh, k, v, slots, *cache)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    R.paged_q4_read(sh, slots, *cache, ko, vo)
    kq, vq = (O.values(*O.quantise(f64(t))) for t in (k, v))
    np.testing.assert_array_equal(f64(ko), kq)
    np.testing.assert_array_equal(f64(vo), vq)
    o, lse = torch.empty_like(q), torch.empty(5, H, device="cuda")
    R.paged_q4_attention(sh, q, *cache, torch.tensor([[P - 1]], dtype=torch.int32, device="cuda"),
                         torch.tensor([0, 5], dtype=torch.int32, device="cuda"),
                         torch.tensor([4005], dtype=torch.int32, device="cuda"), 0.1, o, lse, R.alloc_paged_q4_workspace(sh))
    kf, vf = np.zeros((2, 1, s, H, D))  # (the tokens before read as zeros)
    kf[0, 4000:4005], vf[0, 4000:4005] = kq, vq
    ref = P_.attention(f64(q), kf, vf, np.zeros((1, 1), np.int32), np.array([0, 5]), np.array([4005]), 0.1, 5)
    compare(o, lse, ref + (2.0 ** -39 * 0.1 * 8 * 8 * D, 5 * 2.0 ** -36 * 8), "bf16")


def test_a_wait_that_runs_out_is_reported():
    """A CTA that hands out no work: its waits end by their limit, and the workspace is marked."""
    for io in ("bf16", "f32"):
        x = build([(1, 900)], 2, 1, 64, 16, io, 24)
        R.rglru_debug_lookback(10000, 0)
        try:
            _, _, ws = attend(x, 0.1)
            assert R.rglru_sync_status(ws) == R.ERR_TIMEOUT
        finally:
            R.rglru_debug_lookback(0, -1)
        o, L, ws = attend(x, 0.1)
        assert R.rglru_sync_status(ws) == R.OK
        compare(o, L, expect(x, 0.1), io)


@pytest.mark.parametrize("io,lens,Hq", [("bf16", [(40, 900)], 2), ("bf16", [(600, 900)], 4), ("f32", [(40, 900)], 2)])
def test_a_wait_that_runs_out_is_reported_with_many_rows(io, lens, Hq):
    x = build(lens, Hq, 1, 64, 16, io, 25)
    R.rglru_debug_lookback(10000, 0)
    try:
        _, _, ws = attend(x, 0.1)
        assert R.rglru_sync_status(ws) == R.ERR_TIMEOUT
    finally:
        R.rglru_debug_lookback(0, -1)
    o, L, ws = attend(x, 0.1)
    assert R.rglru_sync_status(ws) == R.OK
    compare(o, L, expect(x, 0.1), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_steps_replayed_from_a_graph(io):
    """plan, write, attention, a fork with its copies and a release, over a cache in 4 bits, captured once and
    replayed with other lengths: each request's output is that over its own tokens as they are held."""
    dt, N, Hq, Hkv, D, s, width, P, T = DT[io], 3, 4, 2, 64, 8, 8, 24, 13
    z = lambda *n, dtype=torch.int32: torch.zeros(*n, dtype=dtype, device="cuda")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    new, lens, state, holders = z(N), z(N), i32([5, P, 0]), z(P)
    ring = i32(np.random.default_rng(1).permutation(P))
    table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
    cu, pos, slots = z(N + 1), z(T), z(T, dtype=torch.int64)
    q, o = (z(T, Hq, D, dtype=dt) for _ in range(2))
    k, v = (z(T, Hkv, D, dtype=dt) for _ in range(2))
    lse = z(T, Hq, dtype=torch.float32)
    sh = R.make_paged_shape(N, T, Hq, Hkv, D, P, s, width, io=dt, window=20)
    cache = R.alloc_paged_q4_cache(sh)
    for c in cache[1::2]:
        c.view(torch.uint8).fill_(0x7f)
    ws, pages_ws = R.alloc_paged_q4_workspace(sh), R.alloc_paged_pages_workspace(sh)
    parents, children, moves, end = i32([-1]), i32([-1]), z(1, 2), z(N)

    def step():
        R.paged_release(sh, z0, end, table, holders, ring, state, table, holders, state, pages_ws)
        R.paged_fork(sh, parents, children, table, lens, holders, ring, state, table, lens, holders, moves, state)
        R.paged_copy(sh, moves, *cache)
        R.paged_plan(sh, lens, new, ring, state, table, cu, lens, pos, slots, state)
        R.paged_q4_write(sh, k, v, slots, *cache)
        R.paged_q4_attention(sh, q, *cache, table, cu, lens, 0.125, o, lse, ws)

    z0 = z(N)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()   # warm-up: nothing new
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    rng = np.random.default_rng(2)
    seqs = [[np.zeros((0, Hkv, D))] * 2 for _ in range(N)]
    for news, fork, ended in (([5, 0, 7], None, []), ([1, 0, 1], (0, 1), []), ([4, 3, 0], None, []), ([1, 1, 1], (0, 2), [2]),
                              ([0, 10, 2], None, []), ([1, 1, 1], (2, 0), [0]), ([3, 0, 8], None, [1])):
        end.copy_(i32([-(-len(seqs[n][0]) // s) if n in ended else 0 for n in range(N)]))
        for n in ended:
            lens[n] = 0
            seqs[n] = [np.zeros((0, Hkv, D))] * 2
        for t, x in zip((parents, children), fork or (-1, -1)):
            t.fill_(x)
        if fork:
            seqs[fork[1]] = list(seqs[fork[0]])
        new.copy_(i32(news))
        for t, H in ((q, Hq), (k, Hkv), (v, Hkv)):
            t.copy_(torch.from_numpy(rng.standard_normal((T, H, D))))
        graph.replay()
        at = 0
        for n, m in enumerate(news):
            held = [O.values(*O.quantise(f64(t)[at:at + m])) if m else np.zeros((0, Hkv, D)) for t in (k, v)]
            seqs[n] = [np.concatenate([a, b]) for a, b in zip(seqs[n], held)]
            if m:
                L = len(seqs[n][0])
                ref = P_.attention(f64(q)[at:at + m], seqs[n][0][None], seqs[n][1][None], np.zeros((1, 1), np.int32), np.array([0, m]),
                                   np.array([L]), 0.125, 20)
                compare(o[at:at + m], lse[at:at + m], ref + (2.0 ** -39 * 0.125 * 8 * 8 * D, L * 2.0 ** -36 * 8), io)
            at += m
        assert int(state[2]) == 0 and lens.tolist() == [len(x[0]) for x in seqs]
    assert R.rglru_sync_status(ws) == R.OK
