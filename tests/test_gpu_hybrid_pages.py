"""The serving example says so when any of its steps wanted pages that it did not get."""
import pytest
import torch

from test_gpu_hybrid_example import load

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("later", [0, 1, 3])
def test_pages_short_in_an_earlier_step_are_reported(later):
    """One page too few in the first step; the later ones stay within the pages that the request counts."""
    E = load()
    model = E.HybridStack(W=256, gate_blocks=2, heads=2, head_dim=64, window=40, pairs=1, io=torch.float32)
    server = E.Server(model, 1, pages=2, page_size=8, longest=64)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    server.step(torch.zeros(17, model.W, device="cuda"), i32([17]))
    for _ in range(later):
        server.step(torch.zeros(1, model.W, device="cuda"), i32([1]), decode=True)
    with pytest.raises(RuntimeError, match="short of 1 page"):
        server.check()


def test_enough_pages_raise_nothing():
    E = load()
    model = E.HybridStack(W=256, gate_blocks=2, heads=2, head_dim=64, window=40, pairs=1, io=torch.float32)
    server = E.Server(model, 1, pages=3, page_size=8, longest=64)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    server.step(torch.zeros(17, model.W, device="cuda"), i32([17]))
    server.step(torch.zeros(1, model.W, device="cuda"), i32([1]), decode=True)
    server.check()
