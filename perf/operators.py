"""The paged-cache operators as measured workloads: the plan that turns request lengths into a block table and slots
(`paged_plan`), the write of new keys and values into their slots (`paged_kv_write`), and the attention of the new tokens over
the paged cache (`paged_attention`).

Where `own` is false, `run` computes them in elementary torch operations in 32 bits; where it is true, through librglru.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # The first thing of every decode step: one new token for each of a few requests.
        {"name": "plan-decode-8", "op": "plan", "N": 8, "q_lo": 1, "q_hi": 1, "c_lo": 90, "c_hi": 2000, "page": 16},
        # The same on a full server.
        {"name": "plan-decode-512", "op": "plan", "N": 512, "q_lo": 1, "q_hi": 1, "c_lo": 16, "c_hi": 8000, "page": 16},
        # A bulk step (offline scoring): many ragged chunks at once, some requests with nothing new.
        {"name": "plan-chunks-1024", "op": "plan", "N": 1024, "q_lo": 0, "q_hi": 513, "c_lo": 0, "c_hi": 4096, "page": 32},
        # A decode step's keys and values for one layer of a 64-request batch.
        {"name": "write-decode-64", "op": "write", "T": 64, "Hkv": 4, "D": 128, "page": 16, "type": "bf16", "fused": True,
         "spare": 0},
        # A prefill's keys and values, read as slices of the fused projection's output.
        {"name": "write-prefill-16384", "op": "write", "T": 16384, "Hkv": 8, "D": 128, "page": 16, "type": "bf16",
         "fused": True, "spare": 0},
        # A padded float32 chunk: the last rows have no slot.
        {"name": "write-f32-3001", "op": "write", "T": 3001, "Hkv": 2, "D": 96, "page": 64, "type": "f32", "fused": False,
         "spare": 13},
        # One request's next token, multi-query heads: latency.
        {"name": "attend-decode-1", "op": "attend", "N": 1, "ones": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 1000, "kv_hi": 1000,
         "Hq": 16, "Hkv": 1, "D": 128, "page": 16, "window": 0, "type": "bf16"},
        # A full server's next tokens, grouped heads, contexts from short to long: the cache's bandwidth.
        {"name": "attend-decode-256", "op": "attend", "N": 256, "ones": 256, "q_lo": 1, "q_hi": 1, "kv_lo": 64,
         "kv_hi": 8192, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "window": 0, "type": "bf16"},
        # A local-attention layer between recurrent ones: ten query heads of 256 on one key head, a window of 2048.
        {"name": "attend-window-128", "op": "attend", "N": 128, "ones": 128, "q_lo": 1, "q_hi": 1, "kv_lo": 500,
         "kv_hi": 32768, "Hq": 10, "Hkv": 1, "D": 256, "page": 32, "window": 2048, "type": "bf16"},
        # Two long prompts from nothing: the tensor cores.
        {"name": "attend-prefill-8192", "op": "attend", "N": 2, "ones": 0, "q_lo": 8192, "q_hi": 8192, "kv_lo": 8192,
         "kv_hi": 8192, "Hq": 16, "Hkv": 4, "D": 128, "page": 64, "window": 0, "type": "bf16"},
        # A step of chunked prefill: four chunks of prompts among twenty decoding requests.
        {"name": "attend-mixed-24", "op": "attend", "N": 24, "ones": 20, "q_lo": 300, "q_hi": 777, "kv_lo": 900,
         "kv_hi": 8192, "Hq": 16, "Hkv": 2, "D": 128, "page": 16, "window": 0, "type": "bf16"},
        # Drafted tokens and short chunks in float32.
        {"name": "attend-f32-5", "op": "attend", "N": 5, "ones": 1, "q_lo": 5, "q_hi": 200, "kv_lo": 201, "kv_hi": 3000,
         "Hq": 8, "Hkv": 2, "D": 64, "page": 16, "window": 0, "type": "f32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attend", "attend", "attend"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "plan":
        N = _log(rng, 1, 1024)
        q_hi = rng.choice([1, _log(rng, 1, 513)])
        return {"op": op, "N": N, "q_lo": min(q_hi, rng.choice([0, 1])), "q_hi": q_hi, "c_lo": rng.choice([0, 1, 90]),
                "c_hi": _log(rng, 100, 8000), "page": page}
    if op == "write":
        D = rng.choice([64, 80, 96, 128, 192, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        most = 16384 * 8 * 128 * 2 // (Hkv * D * (2 if kind == "bf16" else 4))
        return {"op": op, "T": _log(rng, 1, min(most, 40000)), "Hkv": Hkv, "D": D, "page": page, "type": kind,
                "fused": rng.choice([True, False]), "spare": rng.choice([0, 0, 5])}
    while True:
        N = _log(rng, 1, 256)
        D = rng.choice([64, 80, 96, 128, 128, 192, 256])
        Hkv = rng.choice([1, 1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 10, 16])
        q_hi = rng.choice([1, _log(rng, 2, 8), _log(rng, 8, 4096)])
        kv_hi = max(q_hi + 1, _log(rng, 64, 32768))
        c = {"op": op, "N": N, "ones": rng.choice([0, N // 2, N]), "q_lo": rng.randint(1, q_hi), "q_hi": q_hi,
             "kv_lo": rng.randint(q_hi, kv_hi), "kv_hi": kv_hi, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
             "window": rng.choice([0, 0, 0, _log(rng, 32, 4096)]), "type": kind}
        w = work(c)
        rows = max(q for q, _ in _lengths(c))
        padded = N * rows * Hq * kv_hi
        if (padded <= 2.3e9 and N * kv_hi * Hkv * D <= 2.2e9 and w["bytes"] <= 1.7e9
                and w["flops"] <= (2.2e11 if kind == "bf16" else 2e10)):
            return c


def _spread(lo, hi, n, rng):
    """n whole numbers from lo to hi, evenly spaced in their logarithm, in an order of the generator's."""
    if n == 1:
        return [hi]
    v = [int(round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (n - 1)))) - 1 for i in range(n)]
    v = [min(hi, max(lo, x)) for x in v]
    rng.shuffle(v)
    return v


def _lengths(case):
    """(new, all) tokens of every request: a matter of the case alone, as a server knows them on the host."""
    rng = random.Random(11)
    N = case["N"]
    if case["op"] == "plan":
        q = [case["q_lo"]] * N if case["q_lo"] == case["q_hi"] else _spread(case["q_lo"], case["q_hi"], N, rng)
        c = _spread(case["c_lo"], case["c_hi"], N, rng)
        return [(a, a + b) for a, b in zip(q, c)]
    kv = _spread(case["kv_lo"], case["kv_hi"], N, rng)
    ones = case["ones"]
    q = [1] * ones + (_spread(case["q_lo"], case["q_hi"], N - ones, rng) if N > ones else [])
    rng.shuffle(q)
    return [(min(a, b), b) for a, b in zip(q, kv)]


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    if case["op"] == "plan":
        lens = _lengths(case)
        s = case["page"]
        width = max(-(-kv // s) for _, kv in lens) + 3
        held = [-(-(kv - q) // s) for q, kv in lens]
        need = sum(-(-kv // s) for _, kv in lens) - sum(held)
        P = sum(held) + need + 7
        ids = torch.randperm(P, generator=g, **dev).to(torch.int32)
        # what the requests hold, scattered over the pool; the rest of a row is what earlier requests left there
        table = torch.randint(0, P, (case["N"], width), generator=g, dtype=torch.int32, **dev)
        col = torch.arange(width, **dev)[None, :]
        h = torch.tensor(held, **dev)[:, None]
        at = h.cumsum(0) - h + col
        table = torch.where(col < h, ids[at.clamp(max=P - 1)], table).contiguous()
        free = torch.empty(P, dtype=torch.int32, **dev)
        head, count = seed % P, P - sum(held)
        ring = (head + torch.arange(P, **dev)) % P
        free[ring] = torch.roll(ids, -sum(held))
        T = sum(q for q, _ in lens)
        return {"op": "plan", "page": s, "N": case["N"], "T": T, "P": P, "width": width,
                "cached": torch.tensor([kv - q for q, kv in lens], dtype=torch.int32, **dev),
                "new": torch.tensor([q for q, _ in lens], dtype=torch.int32, **dev),
                "free": free, "free_state": torch.tensor([head, count, 0], dtype=torch.int32, **dev), "table": table,
                "cu": torch.empty(case["N"] + 1, dtype=torch.int32, **dev),
                "kv_lens": torch.empty(case["N"], dtype=torch.int32, **dev),
                "positions": torch.empty(T, dtype=torch.int32, **dev), "slots": torch.empty(T, dtype=torch.int64, **dev),
                "free_out": torch.empty(3, dtype=torch.int32, **dev)}
    dt = TYPES[case["type"]]
    Hkv, D, s = case["Hkv"], case["D"], case["page"]
    if case["op"] == "write":
        T = case["T"]
        P = -(-T // s) + 5
        kv = torch.randn(T, 2 * Hkv, D, generator=g, **dev).to(dt)
        k, v = kv[:, :Hkv], kv[:, Hkv:]
        if not case["fused"]:
            k, v = k.contiguous(), v.contiguous()
        # the tokens fill scattered pages, each page in order
        pages = torch.randperm(P, generator=g, **dev)
        t = torch.arange(T, **dev)
        slots = pages[t // s] * s + t % s
        if case["spare"]:
            slots[max(1, T - case["spare"]):] = -1
        return {"op": "write", "P": P, "k": k, "v": v, "slots": slots, "page": s,
                "k_cache": torch.randn(P, s, Hkv, D, generator=g, **dev).to(dt),
                "v_cache": torch.randn(P, s, Hkv, D, generator=g, **dev).to(dt)}
    lens = _lengths(case)
    N, Hq = case["N"], case["Hq"]
    T = sum(q for q, _ in lens)
    width = max(-(-kv // s) for _, kv in lens)
    used = [-(-kv // s) for _, kv in lens]
    P = sum(used) + 3
    ids = torch.randperm(P, generator=g, **dev).to(torch.int32)
    u = torch.tensor(used, **dev)[:, None]
    col = torch.arange(width, **dev)[None, :]
    table = torch.where(col < u, ids[(u.cumsum(0) - u + col).clamp(max=P - 1)], torch.zeros((), dtype=torch.int32, **dev))
    cu = [0]
    for q, _ in lens:
        cu.append(cu[-1] + q)
    return {"op": "attend", "page": s, "N": N, "T": T, "P": P, "width": width, "Hq": Hq, "Hkv": Hkv, "D": D,
            "window": case["window"], "scale": D ** -0.5, "q_max": max(q for q, _ in lens), "kv_max": max(kv for _, kv in lens),
            "q": torch.randn(T, Hq, D, generator=g, **dev).to(dt),
            "k_cache": torch.randn(P, s, Hkv, D, generator=g, dtype=dt, **dev),
            "v_cache": torch.randn(P, s, Hkv, D, generator=g, dtype=dt, **dev), "table": table.contiguous(),
            "cu": torch.tensor(cu, dtype=torch.int32, **dev), "kv_lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, **dev),
            "o": torch.empty(T, Hq, D, dtype=dt, **dev), "lse": torch.empty(T, Hq, **dev)}


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan, "write": _write, "attend": _attend}[state["op"]](state)


def _run_own(x):
    from linear_recurrent_rnn_gb300 import librglru as R
    if "shape" not in x:  # the handle of a user's program: sizes and, for the attention, its scratch
        if x["op"] == "plan":
            x["shape"] = R.make_paged_shape(x["N"], x["T"], num_pages=x["P"], page_size=x["page"], table_width=x["width"])
        elif x["op"] == "write":
            T, Hkv, D = x["k"].shape
            x["shape"] = R.make_paged_shape(1, T, Hkv, Hkv, D, x["P"], x["page"], 1, io=x["k"].dtype)
        else:
            x["shape"] = R.make_paged_shape(x["N"], x["T"], x["Hq"], x["Hkv"], x["D"], x["P"], x["page"], x["width"],
                                            io=x["q"].dtype, window=x["window"])
            x["workspace"] = R.alloc_paged_workspace(x["shape"])
    if x["op"] == "plan":
        R.paged_plan(x["shape"], x["cached"], x["new"], x["free"], x["free_state"], x["table"], x["cu"], x["kv_lens"],
                     x["positions"], x["slots"], x["free_out"])
        return {n: x[n] for n in ("table", "cu", "kv_lens", "positions", "slots", "free_out")}
    if x["op"] == "write":
        R.paged_kv_write(x["shape"], x["k"], x["v"], x["slots"], x["k_cache"], x["v_cache"])
        return {"k_cache": x["k_cache"], "v_cache": x["v_cache"]}
    R.paged_attention(x["shape"], x["q"], x["k_cache"], x["v_cache"], x["table"], x["cu"], x["kv_lens"], x["scale"], x["o"],
                      x["lse"], x["workspace"])
    return {"o": x["o"], "lse": x["lse"]}


def _plan(x):
    s, N, T, P, width = x["page"], x["N"], x["T"], x["P"], x["width"]
    c, q = x["cached"].long(), x["new"].long()
    head, count = x["free_state"][0].long(), x["free_state"][1].long()
    kv = c + q
    cu = torch.cat([torch.zeros_like(q[:1]), q.cumsum(0)])
    held, after = (c + s - 1) // s, (kv + s - 1) // s
    need = after - held
    off = need.cumsum(0) - need
    col = torch.arange(width, device=c.device)[None, :]
    at = off[:, None] + col - held[:, None]
    fresh = x["free"][((head + at) % P).clamp(min=0)]
    fresh = torch.where(at < count, fresh, torch.full_like(fresh, -1))
    table = torch.where((col >= held[:, None]) & (col < after[:, None]), fresh, x["table"])
    x["table"].copy_(table)
    t = torch.arange(T, device=c.device)
    n = torch.searchsorted(cu, t, right=True) - 1
    pos = c[n] + t - cu[n]
    page = table[n, pos // s].long()
    slots = torch.where(page >= 0, page * s + pos % s, torch.full_like(pos, -1))
    taken = torch.minimum(need.sum(), count)
    free_out = torch.stack([(head + taken) % P, count - taken, need.sum() - taken])
    return {"table": x["table"], "cu": cu.int(), "kv_lens": kv.int(), "positions": pos.int(), "slots": slots,
            "free_out": free_out.int()}


def _write(x):
    P, s, Hkv, D = x["k_cache"].shape
    T = x["slots"].numel()
    # the token that fills each slot (one place more, for tokens without a slot), then a choice slot by slot
    at = torch.where(x["slots"] >= 0, x["slots"], torch.full_like(x["slots"], P * s))
    by = torch.full((P * s + 1,), -1, dtype=torch.int64, device=at.device).scatter(0, at, torch.arange(T, device=at.device))[:-1]
    for new, cache in ((x["k"], x["k_cache"]), (x["v"], x["v_cache"])):
        filled = torch.where((by >= 0)[:, None, None], new[by.clamp(min=0)], cache.view(P * s, Hkv, D))
        cache.copy_(filled.view_as(cache))
    return {"k_cache": x["k_cache"], "v_cache": x["v_cache"]}


def _attend(x):
    s, N, Hq, Hkv, D = x["page"], x["N"], x["Hq"], x["Hkv"], x["D"]
    g, Tq, Tk = Hq // Hkv, x["q_max"], x["kv_max"]
    dev = x["q"].device
    cu, kv = x["cu"].long(), x["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    i, j = torch.arange(Tq, device=dev), torch.arange(Tk, device=dev)
    # padded to the longest request: queries [N, Hkv, g Tq, D], keys and values [N, Hkv, Tk, D]
    row = (cu[:-1, None] + i).clamp(max=x["T"] - 1)
    q = x["q"][row].float().view(N, Tq, Hkv, g, D).permute(0, 2, 3, 1, 4).reshape(N, Hkv, g * Tq, D)
    page = x["table"].long()[:, j // s]
    k = x["k_cache"][page, j % s].float().permute(0, 2, 1, 3)
    v = x["v_cache"][page, j % s].float().permute(0, 2, 1, 3)
    pos = (kv - new)[:, None] + i
    seen = (j <= pos[..., None]) & (i < new[:, None])[..., None]
    if x["window"]:
        seen &= j > pos[..., None] - x["window"]
    logits = torch.matmul(q, k.transpose(-1, -2)).mul_(x["scale"]).view(N, Hkv, g, Tq, Tk)
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    weights = logits.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    o = torch.matmul(weights.view(N, Hkv, g * Tq, Tk), v).view(N, Hkv, g, Tq, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    # back to one row a token
    t = torch.arange(x["T"], device=dev)
    n = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[n]
    o = o.permute(0, 3, 1, 2, 4).reshape(N, Tq, Hq, D)[n, at].to(x["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(N, Tq, Hq)[n, at].contiguous()
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers alone
    x = prepare(case, seed)
    if case["op"] == "write":
        P, s = x["k_cache"].shape[:2]
        keep = x["slots"] >= 0
        to = x["slots"][keep]
        out = {}
        for name in ("k", "v"):
            full = x[name + "_cache"].double()
            full[to // s, to % s] = x[name][keep].double()
            out[name + "_cache"] = full
        return out
    s, g, W = case["page"], case["Hq"] // case["Hkv"], case["window"]
    if work(case)["flops"] > 4e12:
        return None
    o = torch.zeros(x["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(x["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    first = 0
    for n, (new, kv) in enumerate(_lengths(case)):
        for a in range(0, new, 1024):  # a stretch of queries against what it can see
            b = min(new, a + 1024)
            lo = max(0, kv - new + a - W + 1) if W else 0
            j = torch.arange(lo, kv - new + b, device="cuda")
            at = x["table"][n, j // s].long()
            p = torch.arange(kv - new + a, kv - new + b, device="cuda")
            away = p[:, None] - j[None, :]
            hidden = (away < 0) | (away >= W) if W else away < 0
            for h in range(case["Hkv"]):
                K, V = (x[c][at, j % s, h].double() for c in ("k_cache", "v_cache"))
                Q = x["q"][first + a:first + b, h * g:(h + 1) * g].double().transpose(0, 1)
                S = (Q @ K.T * x["scale"]).masked_fill(hidden, -math.inf)
                L = torch.logsumexp(S, -1)
                o[first + a:first + b, h * g:(h + 1) * g] = (torch.exp(S - L[..., None]) @ V).transpose(0, 1)
                lse[first + a:first + b, h * g:(h + 1) * g] = L.T
        first += new
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "plan":
        lens = _lengths(case)
        s = case["page"]
        T = sum(q for q, _ in lens)
        fresh = sum(-(-kv // s) - -(-(kv - q) // s) for q, kv in lens)
        return {"bytes": 16 * case["N"] + 8 * fresh + 12 * T + 28, "flops": 0}
    size = 2 if case["type"] == "bf16" else 4
    if case["op"] == "write":
        return {"bytes": case["T"] * (8 + 4 * case["Hkv"] * case["D"] * size), "flops": 0}
    W, D, Hq, Hkv = case["window"], case["D"], case["Hq"], case["Hkv"]
    keys = pairs = T = 0
    for q, kv in _lengths(case):
        first = kv - q + 1  # keys that the first new token sees, itself among them
        if not W or kv <= W:
            pairs += q * first + q * (q - 1) // 2
        else:
            full = max(0, min(q, kv - W))  # rows whose window is full
            part = q - full
            pairs += full * W + part * first + part * (part - 1) // 2
        keys += min(kv, q + W - 1) if W else kv
        T += q
    return {"bytes": 2 * keys * Hkv * D * size + 2 * T * Hq * D * size + 4 * T * Hq, "flops": 4 * D * pairs * Hq}
