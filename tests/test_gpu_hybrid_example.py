"""The serving example: prompts in chunks and single decode steps, through every paged operator and
the recurrent layer's varlen and step calls, against one step over the whole sequences.

Tolerance (float32 I/O): each call is within 1e-5 of the exact layer (the suite's bound for float32),
the two ways differ by at most twice that a call, and a stack of 4 layers on a residual whose layers
are normalised (gain of order 1 each) passes it on with a gain below 10: 4 x 2 x 1e-5 x 10 = 8e-4."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def load():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_serving.py")
    spec = importlib.util.spec_from_file_location("hybrid_serving", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_chunks_and_decode_steps_agree_with_one_pass():
    E = load()
    model = E.HybridStack(W=256, gate_blocks=2, heads=2, head_dim=64, window=40, pairs=2, io=torch.float32, seed=3)
    lens, N = [70, 1, 33, 100], 4
    g = torch.Generator(device="cuda").manual_seed(4)
    xs = [torch.randn(n + 5, model.W, generator=g, device="cuda") for n in lens]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")

    whole = E.Server(model, N, pages=64, page_size=8, longest=128)
    want = whole.step(torch.cat(xs), i32([n + 5 for n in lens])).split([n + 5 for n in lens])
    whole.check()

    parts = E.Server(model, N, pages=64, page_size=8, longest=128)
    got, done = [[] for _ in lens], [0] * N
    for chunk in (17, 1, 100):
        new = [min(chunk, n - d) for n, d in zip(lens, done)]
        y = parts.step(torch.cat([x[d:d + n] for x, d, n in zip(xs, done, new)]), i32(new)).split(new)
        for r, t in zip(got, y):
            r.append(t)
        done = [d + n for d, n in zip(done, new)]
    assert done == lens
    for i in range(5):
        y = parts.step(torch.stack([x[n + i] for x, n in zip(xs, lens)]), i32([1] * N), decode=True)
        for r, t in zip(got, y):
            r.append(t[None])
    parts.check()
    assert parts.lens.tolist() == whole.lens.tolist()
    for a, b in zip(got, want):
        a = torch.cat(a)
        assert torch.isfinite(a).all()
        assert float(((a - b).abs() / b.abs().clamp(min=1)).max()) <= 8e-4


def test_example_runs(capsys):
    load().main()
    assert "us a step" in capsys.readouterr().out
