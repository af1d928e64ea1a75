"""What the Python calls of the cache in 4 bits and of pages that come and go refuse before anything is
launched, tensor by tensor, and the streams that they use.  (Refusals of the C calls: test_paged_q4_abi.py,
test_paged_pages_abi.py.)"""
import pytest
import torch

from linear_recurrent_rnn_gb300 import librglru as R

pytestmark = pytest.mark.gpu

N, T, HQ, HKV, D, P, S, W, M = 2, 3, 4, 2, 64, 8, 16, 4, 3


def zeros(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def shape():
    return R.make_paged_shape(N, T, HQ, HKV, D, P, S, W, R.BF16)


def arguments(call):
    b = torch.bfloat16
    table, ring, state, holders = zeros(N, W), zeros(P), zeros(3), zeros(P)
    if call is R.paged_fork:
        return dict(parents=zeros(M) - 1, children=zeros(M) - 1, block_table=table, kv_lens=zeros(N), holders=holders,
                    free_pages=ring, free_state=state, block_table_out=zeros(N, W), kv_lens_out=zeros(N),
                    holders_out=zeros(P), moves=zeros(M, 2), free_state_out=zeros(3))
    if call is R.paged_release:
        return dict(first_pages=zeros(N), end_pages=zeros(N), block_table=table, holders=holders, free_pages=ring,
                    free_state=state, block_table_out=zeros(N, W), holders_out=zeros(P), free_state_out=zeros(3),
                    workspace=R.alloc_paged_pages_workspace(shape()))
    if call is R.paged_compact:
        return dict(kv_lens=zeros(N), block_table=table, holders=holders, block_table_out=zeros(N, W),
                    holders_out=zeros(P), free_pages=ring, free_state_out=zeros(3), moves=zeros(P // 2, 2),
                    workspace=R.alloc_paged_pages_workspace(shape()))
    kc, ks, vc, vs = R.alloc_paged_q4_cache(shape())
    cache = dict(k_codes=kc, k_scales=ks, v_codes=vc, v_scales=vs)
    if call is not R.paged_q4_attention:
        rows = dict(k=zeros(T, HKV, D, dtype=b), v=zeros(T, HKV, D, dtype=b), slots=zeros(T, dtype=torch.int64))
        return dict(rows, **cache)
    return dict(q=zeros(T, HQ, D, dtype=b), **cache, block_table=table, cu_seqlens=zeros(N + 1), kv_lens=zeros(N),
                scale=0.125, o=zeros(T, HQ, D, dtype=b), lse=zeros(T, HQ, dtype=torch.float32),
                workspace=R.alloc_paged_q4_workspace(shape()))


CALLS = [R.paged_fork, R.paged_release, R.paged_compact, R.paged_q4_write, R.paged_q4_read, R.paged_q4_attention]
CODES = " k_codes k_scales v_codes v_scales"
TENSORS = [(c, n) for c, names in (
    (R.paged_fork, "parents children block_table kv_lens holders free_pages free_state block_table_out kv_lens_out "
                   "holders_out moves free_state_out"),
    (R.paged_release, "first_pages end_pages block_table holders free_pages free_state block_table_out holders_out "
                      "free_state_out workspace"),
    (R.paged_compact, "kv_lens block_table holders block_table_out holders_out free_pages free_state_out moves workspace"),
    (R.paged_q4_write, "k v slots" + CODES), (R.paged_q4_read, "k v slots" + CODES),
    (R.paged_q4_attention, "q block_table cu_seqlens kv_lens o lse workspace" + CODES)) for n in names.split()]


def every_other(t):
    raw = t.view(torch.uint8) if t.element_size() == 1 else t
    return torch.cat([raw, raw], -1).view(t.dtype)[..., ::2]


@pytest.mark.parametrize("call", CALLS)
def test_right_arguments_are_taken(call):
    call(shape(), **arguments(call))
    torch.cuda.synchronize()


@pytest.mark.parametrize("call,name", TENSORS)
def test_wrong_tensors_are_refused_by_name(call, name):
    a = arguments(call)
    t = a[name]
    longer = torch.zeros(t.shape[0] + 1, *t.shape[1:], dtype=t.dtype, device="cuda")
    wrong = {"on the host": t.cpu(), "shorter": longer[:max(t.shape[0] - 1, 0)], "every other element": every_other(t)}
    if name != "workspace":  # (its type and shape are free)
        wrong["another type"] = t.to(torch.float64)
        wrong["another rank"] = t[None]
        if name not in ("parents", "children"):
            wrong["longer"] = longer
    before = R.rglru_kernel_launches()
    for why, x in wrong.items():
        # (a fork's children are as many as its parents: either may be named)
        with pytest.raises(ValueError, match="^(parents|children|moves): " if name in ("parents", "children") else f"^{name}: "):
            call(shape(), **dict(a, **{name: x}))
            pytest.fail(why)
    with pytest.raises(TypeError, match=f"^{name}: "):
        call(shape(), **dict(a, **{name: 5}))
    assert R.rglru_kernel_launches() == before


def test_wrong_moves_and_caches_are_refused():
    c = zeros(P, S, HKV, D, dtype=torch.bfloat16)
    moves = zeros(M, 2) - 1
    R.paged_copy(shape(), moves, c)
    before = R.rglru_kernel_launches()
    for x in (moves.cpu(), moves.long(), moves.flatten(), every_other(moves)):
        with pytest.raises(ValueError, match="^moves: "):
            R.paged_copy(shape(), x, c)
    for x in (c.cpu(), c[:-1], c[:1].expand(P, -1, -1, -1)):
        with pytest.raises((ValueError, R.RglruError)):
            R.paged_copy(shape(), moves, c, x)
    with pytest.raises(TypeError):
        R.paged_copy(shape(), moves, c, 3)
    assert R.rglru_kernel_launches() == before


@pytest.mark.parametrize("call", CALLS)
def test_wrong_shapes_and_scales_are_refused(call):
    a = arguments(call)
    before = R.rglru_kernel_launches()
    with pytest.raises(TypeError):
        call((N, T, HQ, HKV, D, P, S, W, R.BF16, 0), **a)
    if call is R.paged_q4_attention:
        with pytest.raises(TypeError):
            call(shape(), **dict(a, scale="1"))
        with pytest.raises(R.RglruError):
            call(shape(), **dict(a, scale=float("nan")))
    assert R.rglru_kernel_launches() == before


def test_a_workspace_for_fewer_rows_is_refused():
    """Scratch grows with the rows of a row tile: one made for single tokens does not serve long chunks."""
    one, many = (R.make_paged_shape(1, t, 16, 1, 128, 64, 16, 64) for t in (1, 512))
    small = R.alloc_paged_q4_workspace(one)
    assert small.numel() < R.paged_q4_attention_workspace_bytes(many)
    q = zeros(512, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="^workspace: "):
        R.paged_q4_attention(many, q, *R.alloc_paged_q4_cache(many), zeros(1, 64), zeros(2), zeros(1), 0.1, q.clone(), None, small)


@pytest.mark.parametrize("given", [False, True])
def test_current_and_given_streams_order_the_calls(given):
    """The calls run on the current stream, or on the one given: each sees what that stream did before."""
    sh = shape()
    a = arguments(R.paged_q4_write)
    a["slots"].copy_(torch.tensor([3, 40, 127]))
    b = dict(a, k=zeros(T, HKV, D, dtype=torch.bfloat16), v=zeros(T, HKV, D, dtype=torch.bfloat16))
    forks, rel, comp = (arguments(c) for c in (R.paged_fork, R.paged_release, R.paged_compact))
    att = dict(arguments(R.paged_q4_attention), **{n: a[n] for n in CODES.split()})
    moves = zeros(1, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()

    def calls(stream):
        R.paged_q4_write(sh, **a, stream=stream)
        R.paged_copy(sh, moves, a["k_codes"], a["k_scales"], stream=stream)   # page 0 to page 1
        R.paged_q4_read(sh, **b, stream=stream)
        R.paged_fork(sh, **forks, stream=stream)
        R.paged_release(sh, **rel, stream=stream)
        R.paged_compact(sh, **comp, stream=stream)
        R.paged_q4_attention(sh, **att, stream=stream)

    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)  # the calls come before this ends, unless on this stream
        a["k"].fill_(6.0)
        a["v"].fill_(3.0)
        moves.copy_(torch.tensor([[0, 1]]))
        forks["kv_lens"].fill_(5)
        forks["parents"][:1].fill_(0)
        forks["children"][:1].fill_(1)
        rel["holders"].fill_(2)
        comp["kv_lens"].fill_(4)
        att["q"].fill_(1.0)
        att["cu_seqlens"].copy_(torch.tensor([0, 1, 1]))
        att["kv_lens"].copy_(torch.tensor([4, 0]))
        if not given:
            calls(None)
    if given:
        calls(s)
    torch.cuda.synchronize()
    assert (b["k"] == 6.0).all() and (b["v"] == 3.0).all()
    assert (a["k_codes"][1, 3] == a["k_codes"][0, 3]).all() and a["k_codes"][1, 3].any()
    assert int(forks["kv_lens_out"][1]) == 5 and (rel["holders_out"] == 2).all()
    assert int(comp["free_state_out"][1]) == P - 1  # both rows hold page 0
    # four keys, one of them 6 and its value 3 where the others are 0: softmax of [0, 0, 0, 0.125 * 6 * D]
    assert (att["o"][0].float() - 3.0).abs().max() < 0.02 and not att["o"][1:].any()


def test_a_graph_and_direct_calls_take_turns_on_a_workspace():
    """Two captured graphs and direct calls of other sizes share a workspace on a stream, and none changes what
    another gives."""
    g = torch.Generator(device="cuda").manual_seed(3)
    shapes = [R.make_paged_shape(n, t, 8, 2, 128, 64, 16, 16) for n, t in ((3, 3), (2, 400))]
    ws = max((R.alloc_paged_q4_workspace(sh) for sh in shapes), key=lambda w: w.numel())
    runs = []
    for sh, (n, t) in zip(shapes, ((3, 3), (2, 400))):
        cache = R.alloc_paged_q4_cache(sh)
        kv = [torch.randn(64 * 16, 2, 128, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2)]
        whole = R.make_paged_shape(1, 64 * 16, 8, 2, 128, 64, 16, 16)
        R.paged_q4_write(whole, *kv, torch.arange(64 * 16, device="cuda"), *cache)
        q = torch.randn(t, 8, 128, device="cuda", generator=g).to(torch.bfloat16)
        table = torch.randperm(64, device="cuda", generator=g)[:n * 16].to(torch.int32).view(n, 16)
        cu = torch.arange(n + 1, device="cuda", dtype=torch.int32) * (t // n)
        runs.append(dict(shape=sh, q=q, cache=cache, rest=(table, cu, zeros(n) + 250, 0.09), o=torch.zeros_like(q)))

    def attend(r, o):
        R.paged_q4_attention(r["shape"], r["q"], *r["cache"], *r["rest"], o, None, ws)
        return o

    want = [attend(r, torch.zeros_like(r["q"])).clone() for r in runs]
    graphs = []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attend(r, r["o"])
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 0, 1):
        runs[turn]["o"].fill_(5.0)
        graphs[turn].replay()
        other = attend(runs[1 - turn], torch.zeros_like(runs[1 - turn]["q"]))
        assert torch.equal(runs[turn]["o"], want[turn]) and torch.equal(other, want[1 - turn])
    assert R.rglru_sync_status(ws) == R.OK


def test_calls_on_two_streams_at_once():
    """Steps of two servers at once, each with a stream and scratch of its own, give what they give alone."""
    g = torch.Generator(device="cuda").manual_seed(4)

    def server(n, t, kv, dtype):
        sh = R.make_paged_shape(n, n * t, 8, 2, 128, 256, 16, 64, dtype, 300)
        cache = R.alloc_paged_q4_cache(sh)
        kept = [torch.randn(256 * 16, 2, 128, device="cuda", generator=g).to(dtype) for _ in range(2)]
        fill = R.make_paged_shape(1, 256 * 16, 8, 2, 128, 256, 16, 64, dtype)
        q = torch.randn(n * t, 8, 128, device="cuda", generator=g).to(dtype)
        table = torch.randint(0, 256, (n, 64), device="cuda", generator=g, dtype=torch.int32)
        cu = torch.arange(n + 1, device="cuda", dtype=torch.int32) * t
        holders, ring, state = zeros(256), zeros(256), zeros(3)
        first, end = zeros(n), zeros(n) + 30
        ws, pages = R.alloc_paged_q4_workspace(sh), R.alloc_paged_pages_workspace(sh)
        slots = torch.arange(256 * 16, device="cuda")
        outs = [torch.zeros_like(q), torch.zeros_like(table), torch.zeros_like(ring), torch.zeros_like(state)]

        def step(stream):
            R.paged_q4_write(fill, *kept, slots, *cache, stream=stream)
            R.paged_q4_attention(sh, q, *cache, table, cu, zeros_kv, 0.09, outs[0], None, ws, stream=stream)
            R.paged_release(sh, first, end, table, holders, outs[2], state, outs[1], holders_out, outs[3], pages, stream=stream)
        zeros_kv, holders_out = zeros(n) + kv, zeros(256)
        return step, outs, ws

    servers = [server(100, 1, 900, torch.bfloat16), server(3, 150, 1000, torch.float32), server(4, 200, 700, torch.bfloat16)]
    torch.cuda.synchronize()
    want = []
    for step, outs, _ in servers:
        step(None)
        torch.cuda.synchronize()
        want.append([o.clone() for o in outs])
        for o in outs:
            o.zero_()
    streams = [torch.cuda.Stream() for _ in servers]
    torch.cuda.synchronize()
    for _ in range(5):
        for (step, _, _), stream in zip(servers, streams):
            step(stream)
    torch.cuda.synchronize()
    for (_, outs, ws), w in zip(servers, want):
        assert R.rglru_sync_status(ws) == R.OK
        for a, b in zip(outs, w):
            assert torch.equal(a, b)
