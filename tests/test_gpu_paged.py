"""GPU parity of the paged cache (include/paged_attn.h) with the float64 oracle: the plan and the
write exactly, the attention element by element.

Tolerances of the attention, from its arithmetic on inputs taken as stored.  With
A = sum_j p_j |v_j| (the weighted mean of |v|) and B = max_j sum_d |scale q_d k_jd|:
  scores: float32 sums of D products, at most 2^-20 B off (D = 256 terms; an accumulator that
  truncates loses up to 2^-23 of the running magnitude at each of 16 steps); the exponent's
  argument is rounded to 2^-23 of it, its function to 2^-22.  So lse is off by at most
  e = 2^-20 B + 2^-21 max(1, |lse|), and o by 2 e A + 2^-20 A (weights, and float32 sums);
  with bf16 I/O the weights are rounded to bf16, a significand of 8 bits and so a unit roundoff
  of 2^-8 (2^-8 A), and so is the output (half its spacing, at most 2^-8 |o|)."""
import numpy as np
import pytest
import torch

from helpers import half_ulp_bf16
from oracle import paged as O
from linear_recurrent_rnn_gb300 import librglru as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.detach().double().cpu().numpy()


def layout_cache(P, s, H, D, dt, kind):
    """A [P, s, H, D] view, NaN everywhere: contiguous, head by head, or every other page block of
    an interleaved key/value buffer."""
    nan = float("nan")
    if kind == "nhd":
        return torch.full((P, s, H, D), nan, dtype=dt, device="cuda")
    if kind == "hnd":
        return torch.full((P, H, s, D), nan, dtype=dt, device="cuda").transpose(1, 2)
    return torch.full((P, 2, s, H, D), nan, dtype=dt, device="cuda")[:, 1]


def build(lens, Hq, Hkv, D, s, io, seed, layout="nhd", fused=False, spare_rows=0, k_scale=1.0):
    """Requests of (new, all) tokens in scattered pages of a cache that is NaN wherever no request
    has a token, with garbage in the table past each request's pages."""
    rng = np.random.default_rng(seed)
    dt = DT[io]
    N = len(lens)
    used = [-(-kv // s) for _, kv in lens]
    P = sum(used) + 3
    width = max(used + [1]) + 2
    ids = rng.permutation(P)
    table = rng.choice([-1, 0, P - 1, P, 2 ** 30], size=(N, width)).astype(np.int32)
    kc, vc = (layout_cache(P, s, Hkv, D, dt, layout) for _ in range(2))
    at = 0
    for n, (_, kv) in enumerate(lens):
        table[n, :used[n]] = ids[at:at + used[n]]
        at += used[n]
        if kv:
            j = np.arange(kv)
            pg = torch.from_numpy(table[n, j // s].astype(np.int64)).cuda()
            off = torch.from_numpy(j % s).cuda()
            for c, f in ((kc, k_scale), (vc, 1.0)):
                c[pg, off] = torch.from_numpy(rng.standard_normal((kv, Hkv, D)) * f).to(dt).cuda()
    T = sum(q for q, _ in lens) + spare_rows
    qkv = torch.from_numpy(rng.standard_normal((T, Hq + 2 * Hkv, D))).to(dt).cuda()
    q = qkv[:, :Hq] if fused else qkv[:, :Hq].contiguous()
    cu = np.concatenate([[0], np.cumsum([q_ for q_, _ in lens])]).astype(np.int32)
    return dict(q=q, kc=kc, vc=vc, table=torch.from_numpy(table).cuda(), cu=torch.from_numpy(cu).cuda(),
                kv=torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda"),
                dims=(N, T, Hq, Hkv, D, P, s, width), io=io)


def attend(x, scale, window=0, ws=None, o=None, lse=True, stream=None):
    sh = R.make_paged_shape(*x["dims"], io=DT[x["io"]], window=window)
    ws = R.alloc_paged_workspace(sh) if ws is None else ws
    T, Hq, D = x["q"].shape
    o = torch.full((T, Hq, D), 77.0, dtype=x["q"].dtype, device="cuda") if o is None else o
    L = torch.full((T, Hq), 77.0, device="cuda") if lse else None
    R.paged_attention(sh, x["q"], x["kc"], x["vc"], x["table"], x["cu"], x["kv"], scale, o, L, ws, stream)
    return o, L, ws


def expect(x, scale, window=0):
    return O.attention(f64(x["q"]), f64(x["kc"]), f64(x["vc"]), x["table"].cpu().numpy(), x["cu"].cpu().numpy(),
                       x["kv"].cpu().numpy(), scale, window)


def compare(o, L, ref, io):
    ro, rl, av, qk = ref
    live = ~np.isnan(rl)
    o = f64(o)
    assert np.all(o[~live] == 77.0)
    e = 2.0 ** -20 * qk + 2.0 ** -21 * np.maximum(1.0, np.abs(np.where(np.isfinite(rl), rl, 0.0)))
    tol = (2 * e[..., None] + 2.0 ** -20) * av
    if io == "bf16":
        tol = tol + 2.0 ** -8 * av
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
    "odd-width-80": ([(9, 140), (130, 131)], 3, 3, 80, 32, 0),
    "odd-width-8": ([(3, 30)], 2, 1, 8, 8, 0),
    "odd-width-200": ([(5, 150), (70, 70)], 5, 1, 200, 16, 33),
    "prefill-256": ([(150, 150), (90, 300)], 4, 2, 256, 64, 0),
    "group-5": ([(40, 200), (1, 77)], 10, 2, 96, 16, 0),
    "group-64": ([(3, 140), (1, 500)], 64, 1, 128, 16, 0),
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
@pytest.mark.parametrize("layout", ["hnd", "interleaved"])
def test_attention_strided(layout, io):
    """Caches stored head by head or interleaved, queries as slices of a fused projection, the
    output inside a wider buffer, padding rows, no lse."""
    x = build([(20, 150), (1, 40), (3, 3)], 6, 2, 64, 16, io, 5, layout, fused=True, spare_rows=4)
    T = x["q"].shape[0]
    wide = torch.full((T, 9, 64), 77.0, dtype=DT[io], device="cuda")
    o, _, _ = attend(x, 0.2, o=wide[:, 2:8], lse=False)
    assert torch.all(wide[:, :2] == 77.0) and torch.all(wide[:, 8:] == 77.0)
    compare(o, None, expect(x, 0.2), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_large_scores(io):
    """Scores of some hundreds: the running maximum moves far, weights underflow."""
    x = build([(140, 700), (1, 400)], 2, 1, 128, 16, io, 6, k_scale=30.0)
    o, L, _ = attend(x, 128 ** -0.5)
    compare(o, L, expect(x, 128 ** -0.5), io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attention_repeats_bitwise_and_keeps_its_workspace(io):
    """Many CTAs share a request's keys: a second run on the same workspace, and one on another
    stream with its own, give the same bits."""
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
    """Malformed input: entries outside the cache, a length past the table.  Such keys and values
    count as zeros."""
    x = build([(2, 60), (1, 40)], 2, 1, 64, 16, io, 8)
    x["table"][0, 1] = -7
    x["table"][1, 0] = x["dims"][5]
    x["kv"][1] = 16 * x["dims"][7] + 5
    x["table"][1, 1:] = x["table"][0, 0]   # a whole page: all finite
    o, L, _ = attend(x, 0.2)
    compare(o, L, expect(x, 0.2), io)


def test_offsets_out_of_range_stay_in_bounds():
    """cu_seqlens beyond the rows, decreasing and negative: clamped, and no row outside the given
    ones is written."""
    x = build([(3, 20), (2, 30)], 2, 1, 64, 16, "bf16", 9)
    for cu in ([0, 3, 900], [4, 2, -5], [-3, 2 ** 31 - 1, 1]):
        x["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        x["kv"] = torch.tensor([20, -4], dtype=torch.int32, device="cuda")
        buf = torch.full((5 + 64, 2, 64), 77.0, dtype=torch.bfloat16, device="cuda")
        _, _, ws = attend(x, 0.2, o=buf[32:37])
        assert R.rglru_sync_status(ws) == R.OK
        assert torch.all(buf[:32] == 77.0) and torch.all(buf[37:] == 77.0)


def test_long_cache_offsets_pass_32_bits():
    """A cache of over 2^32 elements: the last pages are read and written where they are."""
    P, s, H, D = 4200, 4096, 2, 128
    kc = torch.zeros(P, s, H, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 32
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(5, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(5, H, D, generator=g, device="cuda").bfloat16()
    slots = (P - 1) * s + torch.arange(5, device="cuda") + 4000
    sh = R.make_paged_shape(1, 5, H, H, D, P, s, 1, io=R.BF16, window=5)
    R.paged_kv_write(sh, k, v, slots, kc, vc)
    assert torch.equal(kc[P - 1, 4000:4005], k) and torch.equal(vc[P - 1, 4000:4005], v)
    o, lse = torch.empty_like(q), torch.empty(5, H, device="cuda")
    R.paged_attention(sh, q, kc, vc, torch.tensor([[P - 1]], dtype=torch.int32, device="cuda"),
                      torch.tensor([0, 5], dtype=torch.int32, device="cuda"),
                      torch.tensor([4005], dtype=torch.int32, device="cuda"), 0.1, o, lse,
                      R.alloc_paged_workspace(sh))
    full = np.zeros((1, s, H, D))
    full[0, 4000:4005] = f64(k)
    fv = np.zeros_like(full)
    fv[0, 4000:4005] = f64(v)
    ref = O.attention(f64(q), full, fv, np.zeros((1, 1), np.int32), np.array([0, 5]), np.array([4005]), 0.1, 5)
    compare(o, lse, ref, "bf16")


# ---------------------------------------------------------------- write
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,s,layout", [(1, 1, 8, 8, "nhd"), (7, 3, 80, 16, "hnd"), (300, 2, 128, 64, "nhd"),
                                            (65, 1, 256, 32, "interleaved")])
def test_write_is_exact(T, H, D, s, layout, io):
    rng = np.random.default_rng(T)
    P = -(-T // s) + 2
    kc, vc = (layout_cache(P, s, H, D, DT[io], layout).fill_(0.5) for _ in range(2))
    kv = torch.from_numpy(rng.standard_normal((T, 2 * H, D))).to(DT[io]).cuda()
    k, v = kv[:, :H], kv[:, H:]
    slots = rng.permutation(P * s)[:T].astype(np.int64)
    if T > 5:
        slots[[1, 3, 5]] = [-1, P * s, 2 ** 40]
    sh = R.make_paged_shape(1, T, H, H, D, P, s, 1, io=DT[io])
    want = [O.write(f64(c), f64(r), slots) for c, r in ((kc, k), (vc, v))]
    R.paged_kv_write(sh, k, v, torch.from_numpy(slots).cuda(), kc, vc)
    np.testing.assert_array_equal(f64(kc), want[0])
    np.testing.assert_array_equal(f64(vc), want[1])


# ---------------------------------------------------------------- plan
def run_plan(cached, new, free, state, table, s, tokens, in_place):
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")
    N, width = table.shape
    sh = R.make_paged_shape(N, tokens, num_pages=len(free), page_size=s, table_width=width)
    c, q, st, tb = i32(cached), i32(new), i32(state), i32(table)
    kv = c if in_place else torch.empty_like(c)
    out = st if in_place else torch.empty_like(st)
    cu = torch.empty(N + 1, dtype=torch.int32, device="cuda")
    pos = torch.empty(tokens, dtype=torch.int32, device="cuda")
    slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
    R.paged_plan(sh, c, q, i32(free), st, tb, cu, kv, pos, slots, out)
    return [t.cpu().numpy() for t in (tb, cu, kv, pos, slots, out)]


PLANS = {
    "one": (1, 16, 1, 1, 0),
    "decode": (300, 16, 1, 1, 0),
    "chunks": (33, 8, 0, 40, 0),
    "bulk": (700, 32, 0, 90, 0),
    "many": (8192, 16, 0, 1, 0),
    "pages-run-out": (50, 16, 0, 60, 55),
    "padded": (20, 64, 1, 9, -40),
}


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("name", list(PLANS))
def test_plan_matches_oracle(name, in_place):
    """`less` pages fewer in the ring than wanted (or, negative, padding rows)."""
    N, s, lo, hi, less = PLANS[name]
    rng = np.random.default_rng(N + in_place)
    cached, new = rng.integers(0, 300, N), rng.integers(lo, hi + 1, N)
    if less >= 0 and name != "one":
        cached[0] = new[-1] = 0
    held = -(-cached // s)
    need = int((-(-(cached + new) // s) - held).sum())
    P = int(held.sum()) + need + 5
    ids = rng.permutation(P)
    table = rng.integers(0, P, (N, 300 // s + 4))
    at = 0
    for n in range(N):
        table[n, :held[n]] = ids[at:at + held[n]]
        at += held[n]
    free = np.zeros(P, np.int32)
    head = P - 2
    count = max(0, P - at if less <= 0 else need - less)
    free[(head + np.arange(P - at)) % P] = ids[at:]
    tokens = int(new.sum()) + max(0, -less)
    want = O.plan(cached, new, free, [head, count, 0], table, s, tokens)
    got = run_plan(cached, new, free, [head, count, 0], table, s, tokens, in_place)
    for n, a, b in zip(("table", "cu", "kv_lens", "positions", "slots", "state"), got, want):
        np.testing.assert_array_equal(a, b, err_msg=n)


def test_plan_with_odd_lengths():
    """Negative lengths count as 0, requests past the table's width get what fits, fewer rows than
    new tokens, a head out of range, more free pages said than there are."""
    free = np.arange(12)[::-1].copy()
    table = np.full((4, 3), 11)
    args = ([-5, 20, 70, 0], [9, 40, 3, -2], free, [-13, 100, 9], table, 16)
    want = O.plan(*args, 30)
    for in_place in (False, True):
        got = run_plan(*args, 30, in_place)
        for a, b in zip(got, want):
            np.testing.assert_array_equal(a, b)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_steps_replayed_from_a_graph(io):
    """plan + write + attention captured once (lengths and free pages updated in place) and
    replayed with other lengths each time give what one prefill over every request's whole
    sequence gives, and the pages come off the ring in order."""
    dt, N, Hq, Hkv, D, s, width, P, T = DT[io], 3, 4, 2, 64, 8, 8, 24, 12
    i32 = dict(dtype=torch.int32, device="cuda")
    new = torch.zeros(N, **i32)
    lens = torch.zeros(N, **i32)
    state = torch.tensor([5, P, 0], **i32)
    ring = torch.from_numpy(np.random.default_rng(1).permutation(P)).to(**i32)
    table = torch.full((N, width), -1, **i32)
    cu, pos, slots = torch.zeros(N + 1, **i32), torch.zeros(T, **i32), torch.zeros(T, dtype=torch.int64, device="cuda")
    q, o = (torch.zeros(T, Hq, D, dtype=dt, device="cuda") for _ in range(2))
    k, v = (torch.zeros(T, Hkv, D, dtype=dt, device="cuda") for _ in range(2))
    kc, vc = (layout_cache(P, s, Hkv, D, dt, "nhd") for _ in range(2))
    lse = torch.zeros(T, Hq, device="cuda")
    sh = R.make_paged_shape(N, T, Hq, Hkv, D, P, s, width, io=dt, window=20)
    ws = R.alloc_paged_workspace(sh)

    def step():
        R.paged_plan(sh, lens, new, ring, state, table, cu, lens, pos, slots, state)
        R.paged_kv_write(sh, k, v, slots, kc, vc)
        R.paged_attention(sh, q, kc, vc, table, cu, lens, 0.125, o, lse, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()   # warm-up: no new tokens
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    rng = np.random.default_rng(2)
    seqs = [[[], [], []] for _ in range(N)]   # per request: q, k, v rows
    outs = [[] for _ in range(N)]
    for news in ([5, 0, 7], [1, 1, 1], [4, 3, 0], [1, 1, 1], [0, 10, 2], [1, 1, 1], [3, 0, 8]):
        new.copy_(torch.tensor(news, **i32))
        for t, H in ((q, Hq), (k, Hkv), (v, Hkv)):
            t.copy_(torch.from_numpy(rng.standard_normal((T, H, D))))
        graph.replay()
        at = 0
        for n, m in enumerate(news):
            for r, t in zip(seqs[n], (q, k, v)):
                r.append(t[at:at + m].clone())
            outs[n].append(o[at:at + m].clone())
            at += m
    assert R.rglru_sync_status(ws) == R.OK
    all_q = [[torch.cat(r) for r in x] for x in seqs]
    total = [x[0].shape[0] for x in all_q]
    assert lens.tolist() == total
    pages = sum(-(-t // s) for t in total)
    assert state.tolist() == [(5 + pages) % P, P - pages, 0]
    for n in range(N):
        m = total[n]
        kf, vf = (np.zeros((1, m, Hkv, D)) for _ in range(2))
        kf[0], vf[0] = f64(all_q[n][1]), f64(all_q[n][2])
        ref = O.attention(f64(all_q[n][0]), kf, vf, np.zeros((1, 1), np.int32), np.array([0, m]), np.array([m]), 0.125, 20)
        compare(torch.cat(outs[n]), None, ref, io)
