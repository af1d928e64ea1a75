"""What the Python calls of the paged cache refuse before anything is launched, tensor by tensor,
and the streams that they use.  (Refusals of the C calls: test_paged_abi.py.)"""
import pytest
import torch

from linear_recurrent_rnn_gb300 import librglru as R

pytestmark = pytest.mark.gpu

N, T, HQ, HKV, D, P, S, W = 2, 3, 4, 2, 64, 8, 16, 4


def zeros(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def shape():
    return R.make_paged_shape(N, T, HQ, HKV, D, P, S, W, R.BF16)


def arguments(call):
    b = torch.bfloat16
    if call is R.paged_plan:
        return dict(cached_lens=zeros(N), new_lens=zeros(N), free_pages=zeros(P), free_state=zeros(3),
                    block_table=zeros(N, W), cu_seqlens=zeros(N + 1), kv_lens=zeros(N), positions=zeros(T),
                    slots=zeros(T, dtype=torch.int64), free_state_out=zeros(3))
    cache = dict(k_cache=zeros(P, S, HKV, D, dtype=b), v_cache=zeros(P, S, HKV, D, dtype=b))
    if call is R.paged_kv_write:
        return dict(k=zeros(T, HKV, D, dtype=b), v=zeros(T, HKV, D, dtype=b),
                    slots=zeros(T, dtype=torch.int64), **cache)
    return dict(q=zeros(T, HQ, D, dtype=b), **cache, block_table=zeros(N, W), cu_seqlens=zeros(N + 1),
                kv_lens=zeros(N), scale=0.125, o=zeros(T, HQ, D, dtype=b),
                lse=zeros(T, HQ, dtype=torch.float32), workspace=R.alloc_paged_workspace(shape()))


CALLS = [R.paged_plan, R.paged_kv_write, R.paged_attention]
TENSORS = [(c, n) for c, names in (
    (R.paged_plan, "cached_lens new_lens free_pages free_state block_table cu_seqlens kv_lens positions slots "
                   "free_state_out"),
    (R.paged_kv_write, "k v slots k_cache v_cache"),
    (R.paged_attention, "q k_cache v_cache block_table cu_seqlens kv_lens o lse workspace")) for n in names.split()]


@pytest.mark.parametrize("call", CALLS)
def test_right_arguments_are_taken(call):
    call(shape(), **arguments(call))
    torch.cuda.synchronize()


@pytest.mark.parametrize("call,name", TENSORS)
def test_wrong_tensors_are_refused_by_name(call, name):
    a = arguments(call)
    t = a[name]
    wrong = {"on the host": t.cpu(), "shorter": t[:-1], "every other element": torch.cat([t, t], -1)[..., ::2]}
    if name != "workspace":  # (its type and shape are free)
        wrong["another type"] = t.to(torch.float64)
        wrong["another rank"] = t[None]
        wrong["longer"] = torch.cat([t, t[:1]])
    before = R.rglru_kernel_launches()
    for why, x in wrong.items():
        with pytest.raises(ValueError, match=f"^{name}: "):
            call(shape(), **dict(a, **{name: x}))
            pytest.fail(why)
    with pytest.raises(TypeError, match=f"^{name}: "):
        call(shape(), **dict(a, **{name: 5}))
    assert R.rglru_kernel_launches() == before


@pytest.mark.parametrize("call", CALLS)
def test_wrong_shapes_and_scales_are_refused(call):
    a = arguments(call)
    before = R.rglru_kernel_launches()
    with pytest.raises(TypeError):
        call((N, T, HQ, HKV, D, P, S, W, R.BF16, 0), **a)
    if call is R.paged_attention:
        with pytest.raises(TypeError):
            call(shape(), **dict(a, scale="1"))
        with pytest.raises(R.RglruError):
            call(shape(), **dict(a, scale=float("nan")))
    assert R.rglru_kernel_launches() == before


def test_a_workspace_for_fewer_rows_is_refused():
    """Scratch grows with the rows of a row tile: one made for single tokens does not serve long chunks."""
    one, many = (R.make_paged_shape(1, t, 16, 1, 128, 64, 16, 64) for t in (1, 512))
    b = torch.bfloat16
    small = R.alloc_paged_workspace(one)
    assert small.numel() < R.paged_attention_workspace_bytes(many)
    q, c = zeros(512, 16, 128, dtype=b), zeros(64, 16, 1, 128, dtype=b)
    with pytest.raises(ValueError, match="^workspace: "):
        R.paged_attention(many, q, c, c, zeros(1, 64), zeros(2), zeros(1), 0.1, q.clone(), None, small)


def test_current_and_given_streams_order_the_calls():
    """The calls run on the current stream, or on the one given: each sees what that stream did before."""
    a = arguments(R.paged_kv_write)
    a["slots"].copy_(torch.tensor([3, 40, 127]))
    for given in (False, True):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        a["k_cache"].zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # the write comes before this ends, unless on this stream
            a["k"].fill_(7.0 + given)
            if not given:
                R.paged_kv_write(shape(), **a)
        if given:
            R.paged_kv_write(shape(), **a, stream=s)
        torch.cuda.synchronize()
        flat = a["k_cache"].view(P * S, HKV, D)
        assert (flat[[3, 40, 127]] == 7.0 + given).all()
        assert int((flat != 0).any(-1).any(-1).sum()) == 3


def test_sizes_of_one_take_any_stride():
    """A dimension of one element may have any stride (a column of a larger tensor)."""
    b = torch.bfloat16
    sh = R.make_paged_shape(1, 1, 1, 1, D, 1, S, 1)
    k = torch.randn(4, 3, D, device="cuda").to(b)[2:3, 1:2]
    kc = torch.zeros(2, S, 5, D, dtype=b, device="cuda")[1:2, :, 3:4]
    assert k.stride(1) != 3 * D
    R.paged_kv_write(sh, k, k, torch.tensor([5], device="cuda"), kc, kc.clone())
    assert (kc[0, 5, 0] == k[0, 0]).all() and not kc[0, :5].any() and not kc[0, 6:].any()
