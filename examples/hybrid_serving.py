"""A small hybrid language-model stack served with librglru: recurrent layers (RG-LRU) alternate
with local multi-query attention over a paged cache, for several requests at once.

One step appends any number of new tokens to every request, a chunk of its prompt or the next
token, and needs no length on the host:

    paged_plan                     once a step: offsets, pages, slots, positions
    rglru_fused_forward_varlen     each recurrent layer, states carried from step to step
      (or rglru_step, when every request gets exactly one token)
    paged_kv_write, paged_attention  each attention layer

`python examples/hybrid_serving.py` prefills ragged prompts in chunks, then decodes with the step
captured once in a CUDA graph and replayed.  Weights are random; the projections around the
layers are plain matrix products.
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_recurrent_rnn_gb300 import librglru as R  # noqa: E402


class HybridStack:
    """`pairs` x (recurrent layer, attention layer) of width W, each on a normalised residual."""

    def __init__(self, W=512, gate_blocks=4, heads=4, head_dim=128, window=256, pairs=2, io=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, scale: (torch.randn(*s, generator=g, device="cuda") * scale).to(io)
        self.W, self.nblk, self.Hq, self.D, self.window, self.io = W, gate_blocks, heads, head_dim, window, io
        k = W // gate_blocks
        self.pairs = [{
            "in": r(W, W, scale=W ** -0.5), "out": r(W, W, scale=W ** -0.5),
            "Wa": r(gate_blocks, k, k, scale=k ** -0.5), "Wx": r(gate_blocks, k, k, scale=k ** -0.5),
            "ba": torch.zeros(W, device="cuda"), "bx": torch.zeros(W, device="cuda"),
            # decays exp(-8 softplus(Lambda) / 2) from 0.9 to 0.999 at a half-open gate
            "Lambda": torch.log(torch.expm1(-torch.log(torch.linspace(0.9, 0.999, W, device="cuda")) / 4)),
            "qkv": r(W, (heads + 2) * head_dim, scale=W ** -0.5), "o": r(heads * head_dim, W, scale=W ** -0.5),
        } for _ in range(pairs)]


class Server:
    """The state of `requests` concurrent requests: recurrent states, the paged cache, lengths."""

    def __init__(self, model: HybridStack, requests: int, pages: int, page_size: int = 16, longest: int = 4096):
        m, i32 = model, dict(dtype=torch.int32, device="cuda")
        self.m, self.N, self.page_size = m, requests, page_size
        self.width = -(-longest // page_size)
        self.lens = torch.zeros(requests, **i32)
        self.free_pages = torch.arange(pages, **i32)              # the ring of free pages
        self.free_state = torch.tensor([0, pages, 0], **i32)      # its head, its count, pages wanting in the last step
        self.wanting = torch.zeros(1, **i32)                      # and in all steps
        self.table = torch.full((requests, self.width), -1, **i32)
        self.cu = torch.zeros(requests + 1, **i32)
        self.states = [torch.zeros(requests, m.W, device="cuda") for _ in m.pairs]
        self.cache = [torch.empty(2, pages, page_size, 1, m.D, dtype=m.io, device="cuda") for _ in m.pairs]
        self.buffers = {}

    def _buffers(self, T: int, decode: bool):
        """Shapes and scratch of steps of T rows."""
        if (T, decode) not in self.buffers:
            m = self.m
            shape = R.make_paged_shape(self.N, T, m.Hq, 1, m.D, self.free_pages.numel(), self.page_size, self.width,
                                       io=m.io, window=m.window)
            rec = R.make_shape(self.N if decode else 1, 1 if decode else T, m.W, m.nblk, m.io, m.io, R.CANONICAL)
            self.buffers[T, decode] = (
                shape, R.alloc_paged_workspace(shape), torch.empty(T, dtype=torch.int32, device="cuda"),
                torch.empty(T, dtype=torch.int64, device="cuda"), rec, None if decode else R.alloc_saved(rec))
        return self.buffers[T, decode]

    def step(self, x: torch.Tensor, new: torch.Tensor, decode: bool = False) -> torch.Tensor:
        """Appends new[n] (int32, on the GPU) tokens to request n: x [sum of new, W] are their
        embeddings, packed; returns the stack's output for them.  decode: every new[n] is 1."""
        m = self.m
        shape, ws, positions, slots, rec, saved = self._buffers(x.shape[0], decode)
        R.paged_plan(shape, self.lens, new, self.free_pages, self.free_state, self.table, self.cu, self.lens, positions,
                     slots, self.free_state)
        self.wanting += self.free_state[2]
        angle = positions[:, None] * torch.exp2(torch.arange(m.D // 2, device="cuda") * (-20.0 / m.D))
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]

        def rotate(t):
            a, b = t.float().chunk(2, -1)
            return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(m.io)

        def norm(t):
            f = t.float()
            return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(m.io)

        for p, h, cache in zip(m.pairs, self.states, self.cache):
            u = norm(x) @ p["in"]
            y = torch.empty_like(u)
            if decode:
                R.rglru_step(rec, u, p["Wa"], p["ba"], p["Wx"], p["bx"], p["Lambda"], None, h, y, h)
            else:
                hT = torch.empty_like(h)
                R.rglru_fused_forward_varlen(rec, u, p["Wa"], p["ba"], p["Wx"], p["bx"], p["Lambda"], self.cu, self.N, h,
                                             y, hT, saved)
                h.copy_(hT)
            x = x + y @ p["out"]
            qkv = (norm(x) @ p["qkv"]).view(-1, m.Hq + 2, m.D)
            q, k = rotate(qkv[:, :m.Hq]), rotate(qkv[:, m.Hq:-1])
            R.paged_kv_write(shape, k, qkv[:, -1:], slots, cache[0], cache[1])
            o = torch.empty_like(q)
            R.paged_attention(shape, q, cache[0], cache[1], self.table, self.cu, self.lens, m.D ** -0.5, o, None, ws)
            x = x + o.view(-1, m.Hq * m.D) @ p["o"]
        return x

    def check(self):
        """Raises if a step wanted pages it did not get, or a device wait ran out (synchronises)."""
        if int(self.wanting):
            raise RuntimeError(f"the cache was short of {int(self.wanting)} pages")
        for shape, ws, _, _, _, saved in self.buffers.values():
            for b in (ws,) if saved is None else (ws, saved):
                if R.rglru_sync_status(b) != R.OK:
                    raise RuntimeError("a device wait ran out")


def main():
    torch.cuda.set_device(0)
    model, N, prompts = HybridStack(), 32, [37 * (n % 9) + 5 for n in range(32)]
    server = Server(model, N, pages=2048)
    g = torch.Generator(device="cuda").manual_seed(1)
    chunk, done = 128, [0] * N
    while done != prompts:  # prompts in chunks; requests whose prompt is through wait
        new = [min(chunk, p - d) for p, d in zip(prompts, done)]
        x = torch.randn(sum(new), model.W, generator=g, device="cuda").to(model.io)
        y = server.step(x, torch.tensor(new, dtype=torch.int32, device="cuda"))
        done = [d + n for d, n in zip(done, new)]
    server.check()

    x, ones = torch.empty(N, model.W, dtype=model.io, device="cuda"), torch.ones(N, dtype=torch.int32, device="cuda")
    x.copy_(y[-N:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(server.step(x, ones, decode=True))  # warm-up: a step like any other
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(server.step(x, ones, decode=True))  # (a model would sample and embed a token here)
    torch.cuda.synchronize()
    t, steps = time.perf_counter(), 200
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    server.check()
    total = server.lens.tolist()
    assert total == [p + steps + 1 for p in prompts], total
    print(f"{N} requests, prompts of 5 to {max(prompts)} tokens, {steps} decode steps: {t / steps * 1e6:.0f} us a step "
          f"({2 * len(model.pairs)} layers of width {model.W}), {int(server.free_state[1])} pages free")


if __name__ == "__main__":
    main()
