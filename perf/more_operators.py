"""Further operators of the paged cache as measured workloads: the cache held in 4 bits (`paged_q4_write`, `paged_q4_read`, and the
attention over it, `paged_q4_attention`), and its pages as requests come and go (`paged_fork`, `paged_release`, `paged_compact`, and
`paged_copy`, which moves their contents).

Where `own` is false, `run` computes them in elementary torch operations in 32 bits; where it is true, through librglru.

In 4 bits: 16 neighbouring channels of a head share a scale s, E4M3: the number nearest to max |x| / 6, from 2^-9 to 448 (NaN where one of the
16 is no finite number); each x is held as the number nearest to x / s of 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, ties to the even code.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # A decode step's keys and values for one layer of a 64-request batch.
        {"name": "write4-decode-64", "op": "write", "T": 64, "Hkv": 4, "D": 128, "page": 16, "type": "bf16", "spare": 0},
        # A prefill's keys and values, as slices of the fused projection's output.
        {"name": "write4-prefill-16384", "op": "write", "T": 16384, "Hkv": 8, "D": 128, "page": 16, "type": "bf16", "spare": 0},
        # One request's next token, multi-query heads: latency.
        {"name": "attend4-decode-1", "op": "attend", "N": 1, "ones": 1, "q_lo": 1, "q_hi": 1, "kv_lo": 1000, "kv_hi": 1000,
         "Hq": 16, "Hkv": 1, "D": 128, "page": 16, "window": 0, "type": "bf16"},
        # A full server's next tokens, grouped heads, contexts from short to long: the cache's bandwidth.
        {"name": "attend4-decode-256", "op": "attend", "N": 256, "ones": 256, "q_lo": 1, "q_hi": 1, "kv_lo": 64, "kv_hi": 8192,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "window": 0, "type": "bf16"},
        # A step of chunked prefill: four chunks of prompts among twenty decoding requests.
        {"name": "attend4-mixed-24", "op": "attend", "N": 24, "ones": 20, "q_lo": 300, "q_hi": 777, "kv_lo": 900, "kv_hi": 8192,
         "Hq": 16, "Hkv": 2, "D": 128, "page": 16, "window": 0, "type": "bf16"},
        # Drafted tokens of a local-attention layer in float32: ten query heads of 256 on one key head, a window of 2048.
        {"name": "attend4-window-f32-48", "op": "attend", "N": 48, "ones": 16, "q_lo": 2, "q_hi": 7, "kv_lo": 500, "kv_hi": 16000,
         "Hq": 10, "Hkv": 1, "D": 256, "page": 32, "window": 2048, "type": "f32"},
        # Four answers to one prompt of odd length: its pages are shared, the last one is copied in every layer.
        {"name": "fork-4", "op": "fork", "groups": 1, "each": 4, "len_lo": 1371, "len_hi": 1371, "layers": 8, "Hkv": 1, "D": 128,
         "page": 16, "type": "bf16"},
        # A full server: eight answers to each of 32 prompts.
        {"name": "fork-256", "op": "fork", "groups": 32, "each": 8, "len_lo": 40, "len_hi": 8190, "layers": 8, "Hkv": 8, "D": 128,
         "page": 16, "type": "bf16"},
        # A few requests end.
        {"name": "release-8", "op": "release", "N": 8, "len_lo": 90, "len_hi": 2000, "page": 16, "shared": 0.5, "ended": 1.0},
        # Many end at once, of a pool of hundreds of thousands of pages: half of their prompts were shared.
        {"name": "release-1024", "op": "release", "N": 1024, "len_lo": 16, "len_hi": 16000, "page": 16, "shared": 0.5, "ended": 0.75},
        # A small pool is closed up, all layers' pages moved.
        {"name": "compact-12", "op": "compact", "N": 12, "len_lo": 30, "len_hi": 900, "fill": 0.4, "layers": 2, "Hkv": 2, "D": 64,
         "page": 16, "type": "f32"},
        # A server gives a part of its cache back: what is left lies all over it.
        {"name": "compact-96", "op": "compact", "N": 96, "len_lo": 100, "len_hi": 8000, "fill": 0.5, "layers": 2, "Hkv": 8, "D": 128,
         "page": 16, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend", "fork", "release", "compact"])
    page = rng.choice([8, 16, 32, 64, 128, 256])
    kind = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "write":
        D = rng.choice([64, 96, 128, 192, 256] + ([80] if page > 8 else []))
        Hkv = rng.choice([1, 2, 3, 4, 8])
        most = 16384 * 8 * 128 * 2 // (Hkv * D * (2 if kind == "bf16" else 4))
        return {"op": op, "T": _log(rng, 1, min(most, 40000)), "Hkv": Hkv, "D": D, "page": page, "type": kind,
                "spare": rng.choice([0, 0, 5])}
    if op == "release":
        N = _log(rng, 1, 1024)
        lo, hi = sorted((_log(rng, 1, 16000), _log(rng, 1, 16000)))
        return {"op": op, "N": N, "len_lo": lo, "len_hi": hi, "page": rng.choice([16, 32, 64, 128]), "shared": rng.choice([0.0, 0.3, 0.9]),
                "ended": rng.choice([0.1, 0.5, 1.0])}
    while True:
        if op == "fork":
            lo, hi = sorted((_log(rng, 1, 8190), _log(rng, 1, 8190)))
            c = {"op": op, "groups": _log(rng, 1, 64), "each": rng.randint(1, 16), "len_lo": lo, "len_hi": hi}
        elif op == "compact":
            lo, hi = sorted((_log(rng, 1, 8000), _log(rng, 1, 8000)))
            c = {"op": op, "N": _log(rng, 1, 256), "len_lo": lo, "len_hi": hi, "fill": rng.choice([0.1, 0.5, 0.9, 1.0])}
        if op != "attend":
            c |= {"layers": rng.randint(1, 16), "Hkv": rng.choice([1, 2, 3, 8]), "D": rng.choice([64, 80, 128, 256]), "page": page, "type": kind}
            pool = (2 * c["layers"] * c["Hkv"] * c["D"] * (2 if kind == "bf16" else 4)
                    * _pages(c)[1] * page)
            if pool <= 2.6e9 and work(c)["bytes"] <= 1e9:
                return c
            continue
        N = _log(rng, 1, 256)
        D = rng.choice([64, 96, 128, 128, 192, 256] + ([80] if page > 8 else []))
        Hkv = rng.choice([1, 1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8, 10, 16])
        q_hi = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 8, 2048)])
        kv_hi = max(q_hi + 1, _log(rng, 64, 32768))
        c = {"op": op, "N": N, "ones": rng.choice([0, N // 2, N]), "q_lo": rng.randint(1, q_hi), "q_hi": q_hi,
             "kv_lo": rng.randint(q_hi, kv_hi), "kv_hi": kv_hi, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
             "window": rng.choice([0, 0, 0, _log(rng, 32, 4096)]), "type": kind}
        w = work(c)
        rows = max(q for q, _ in _lengths(c))
        if (N * rows * Hq * kv_hi <= 2.3e9 and N * kv_hi * Hkv * D <= 2.2e9 and w["bytes"] <= 4.8e8
                and w["flops"] <= (7e10 if kind == "bf16" else 1.5e10)):
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
    kv = _spread(case["kv_lo"], case["kv_hi"], N, rng)
    ones = case["ones"]
    q = [1] * ones + (_spread(case["q_lo"], case["q_hi"], N - ones, rng) if N > ones else [])
    rng.shuffle(q)
    return [(min(a, b), b) for a, b in zip(q, kv)]


def _pages(case):
    """(tokens of the requests, pages of the pool)."""
    s = case["page"]
    if case["op"] == "fork":
        lens = _spread(case["len_lo"], case["len_hi"], case["groups"], random.Random(12))
        return lens, sum(-(-x // s) for x in lens) + len(lens) * case["each"] + 9
    lens = _spread(case["len_lo"], case["len_hi"], case["N"], random.Random(12))
    used = sum(-(-x // s) for x in lens)
    return lens, used + 11 if case["op"] == "release" else int(used / case["fill"]) + 3


def _ended(case):
    """How many of the requests are released."""
    return max(1, int(case["N"] * case["ended"]))


# ------------------------------------------------------------------------------------------------ 4 bits, plain
def _quantise(x):
    """x [..., D] in float32 as codes uint8 [..., D / 2] (even channels in the low half) and scales E4M3 [..., D / 16]."""
    g = x.unflatten(-1, (-1, 16))
    size = g.abs()
    top = size.amax(-1, keepdim=True)
    s = (top / 6).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    fine = torch.isfinite(top)
    # the borders between neighbours are products of 4 and 3 bits, exact: at or past a border whose upper side is even, past the others
    code = sum((size > s * b).byte() for b in (0.25, 1.25, 2.5, 5.0)) + sum((size >= s * b).byte() for b in (0.75, 1.75, 3.5))
    code = torch.where(fine, code + 8 * torch.signbit(g).byte(), torch.zeros_like(code)).flatten(-2)
    s = torch.where(fine, s, torch.full_like(s, math.nan))
    return code[..., 0::2] + 16 * code[..., 1::2], s[..., 0].to(torch.float8_e4m3fn)


def _values(codes, scales):
    """What codes and scales stand for, in float32."""
    c = torch.stack([codes % 16, codes // 16], -1).flatten(-2).long()
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    return (table[c].unflatten(-1, (-1, 16)) * scales.float()[..., None]).flatten(-2)


def _empty_q4(P, s, Hkv, D):
    """A cache's codes and scales, page by page and head by head; rows of codes on 16 bytes, rows of scales on 4."""
    c = torch.zeros(P, Hkv, s, -(-D // 32) * 16, dtype=torch.uint8, device="cuda")[..., :D // 2]
    x = torch.zeros(P, Hkv, s, -(-D // 64) * 4, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[..., :D // 16]
    return c.transpose(1, 2), x.transpose(1, 2)


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    return {"write": _prepare_write, "attend": _prepare_attend}.get(case["op"], _prepare_pages)(case, seed, g, dev)


def _prepare_write(case, seed, g, dev):
    dt, T, Hkv, D, s = TYPES[case["type"]], case["T"], case["Hkv"], case["D"], case["page"]
    P = -(-T // s) + 5
    # a head's channels differ in size, as keys' do
    size = torch.exp(torch.randn(2 * Hkv, D, generator=g, **dev) * 0.7)
    kv = (torch.randn(T, 2 * Hkv, D, generator=g, **dev) * size).to(dt)
    pages = torch.randperm(P, generator=g, **dev)  # the tokens fill scattered pages, each page in order
    t = torch.arange(T, **dev)
    slots = pages[t // s] * s + t % s
    if case["spare"]:
        slots[max(1, T - case["spare"]):] = -1
    (kc, ks), (vc, vs) = _empty_q4(P, s, Hkv, D), _empty_q4(P, s, Hkv, D)
    return {"op": "write", "k": kv[:, :Hkv], "v": kv[:, Hkv:], "slots": slots, "k_codes": kc, "k_scales": ks, "v_codes": vc,
            "v_scales": vs, "k_out": torch.zeros(T, Hkv, D, dtype=dt, **dev), "v_out": torch.zeros(T, Hkv, D, dtype=dt, **dev)}


def _prepare_attend(case, seed, g, dev):
    dt, Hkv, D, s = TYPES[case["type"]], case["Hkv"], case["D"], case["page"]
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
    x = {"op": "attend", "page": s, "N": N, "T": T, "P": P, "width": width, "Hq": Hq, "Hkv": Hkv, "D": D, "window": case["window"],
         "scale": D ** -0.5, "q_max": max(q for q, _ in lens), "kv_max": max(kv for _, kv in lens),
         "q": torch.randn(T, Hq, D, generator=g, **dev).to(dt), "table": table.contiguous(),
         "cu": torch.tensor(cu, dtype=torch.int32, **dev), "kv_lens": torch.tensor([kv for _, kv in lens], dtype=torch.int32, **dev),
         "o": torch.empty(T, Hq, D, dtype=dt, **dev), "lse": torch.empty(T, Hq, **dev)}
    for n in "kv":
        codes, scales = _empty_q4(P, s, Hkv, D)
        size = torch.exp(torch.randn(Hkv, 1, D, generator=g, **dev) * 0.3)
        step = max(1, 2 ** 27 // (s * Hkv * D))
        for a in range(0, P, step):  # in stretches: the values in 32 bits are many times the cache
            b = min(P, a + step)
            c, x8 = _quantise(torch.randn(b - a, Hkv, s, D, generator=g, **dev) * size)
            codes[a:b] = c.transpose(1, 2)
            scales.view(torch.uint8)[a:b] = x8.view(torch.uint8).transpose(1, 2)
        x[n + "_codes"], x[n + "_scales"] = codes, scales
    return x


def _prepare_pages(case, seed, g, dev):
    s = case["page"]
    lens, P = _pages(case)
    i32 = dict(dtype=torch.int32, **dev)
    N = len(lens)
    children = case["groups"] * case["each"] if case["op"] == "fork" else 0
    width = max(-(-x // s) for x in lens) + 2
    L = torch.tensor(lens, **dev)
    held = (L + s - 1) // s
    ids = torch.randperm(P, generator=g, **dev).to(torch.int32)
    col = torch.arange(width, **dev)[None, :]
    at = (held.cumsum(0) - held)[:, None] + col
    # what the requests hold, scattered over the pool; the rest of a row is what earlier requests left there
    stale = torch.randint(0, P, (N, width), generator=g, **i32)
    table = torch.where(col < held[:, None], ids[at.clamp(max=P - 1)], stale)
    used = int(sum(-(-x // s) for x in lens))
    head, count = seed % P, P - used
    free = torch.full((P,), -1, **i32)
    free[(head + torch.arange(count, **dev)) % P] = ids[used:]
    x = {"op": case["op"], "page": s, "P": P, "width": width, "free": free, "free_state": torch.tensor([head, count, 0], **i32),
         "free_out": torch.empty(3, **i32), "holders": torch.zeros(P, **i32), "holders_out": torch.empty(P, **i32)}
    if case["op"] == "fork":
        rows = N + children  # the prompts, and rows for their answers
        x["N"] = rows
        x["table"] = torch.cat([table, torch.randint(0, P, (children, width), generator=g, **i32)]).contiguous()
        x["lens"] = torch.cat([L, torch.zeros(children, **dev)]).to(torch.int32)
        x["parents"] = torch.arange(N, **i32).repeat_interleave(case["each"])
        x["children"] = (N + torch.randperm(children, generator=g, **dev)).to(torch.int32)
        x["table_out"], x["lens_out"] = x["table"].clone(), x["lens"].clone()
        x["moves"] = torch.empty(children, 2, **i32)
    elif case["op"] == "release":
        x["N"], x["table"] = N, table.contiguous()
        gone = torch.randperm(N, generator=g, **dev) < _ended(case)
        x["first"] = torch.zeros(N, **i32)
        x["end"] = torch.where(gone, held, torch.zeros_like(held)).to(torch.int32)
        # a request shares the first part of its pages with one or two others that go on
        lead = (held * case["shared"]).long()[:, None]
        other = torch.randint(1, 3, (N, 1), generator=g, **i32).expand(N, width)
        sharing = (col < lead) & (torch.rand(N, 1, generator=g, **dev) < 0.5)
        spare = torch.zeros(P + 1, **i32)
        spare[torch.where(sharing, table, torch.full_like(table, P)).long()] = other
        x["holders"] = spare[:P].contiguous()
    else:
        x["N"], x["table"], x["lens"] = N, table.contiguous(), L.to(torch.int32)
        x["table_out"], x["moves"] = x["table"].clone(), torch.empty(P // 2, 2, **i32)
        spare = torch.zeros(P, **i32)
        spare[ids[:used].long()] = (torch.rand(used, generator=g, **dev) < 0.2).to(torch.int32)
        x["holders"] = spare
    if "layers" in case:
        x["caches"] = [torch.randn(P, s, case["Hkv"], case["D"], generator=g, dtype=TYPES[case["type"]], **dev)
                       for _ in range(2 * case["layers"])]
    return x


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _run_own(state)
    return {"write": _write, "attend": _attend, "fork": _fork, "release": _release, "compact": _compact}[state["op"]](state)


def _run_own(x):
    from linear_recurrent_rnn_gb300 import librglru as R
    if "shape" not in x:  # the handle of a user's program: sizes, and scratch
        if x["op"] == "write":
            T, Hkv, D = x["k"].shape
            P, s = x["k_codes"].shape[:2]
            x["shape"] = R.make_paged_shape(1, T, Hkv, Hkv, D, P, s, 1, io=x["k"].dtype)
        elif x["op"] == "attend":
            x["shape"] = R.make_paged_shape(x["N"], x["T"], x["Hq"], x["Hkv"], x["D"], x["P"], x["page"], x["width"],
                                            io=x["q"].dtype, window=x["window"])
            x["workspace"] = R.alloc_paged_q4_workspace(x["shape"])
        else:
            x["shape"] = R.make_paged_shape(x["N"], 0, num_pages=x["P"], page_size=x["page"], table_width=x["width"])
            x["workspace"] = R.alloc_paged_pages_workspace(x["shape"])
            if x["op"] == "release":
                x["table_out"] = x["table"].clone()  # (the inputs stay as they are, for another pass)
    sh = x["shape"]
    if x["op"] == "write":
        cache = (x["k_codes"], x["k_scales"], x["v_codes"], x["v_scales"])
        R.paged_q4_write(sh, x["k"], x["v"], x["slots"], *cache)
        R.paged_q4_read(sh, x["slots"], *cache, x["k_out"], x["v_out"])
        return {"k": x["k_out"], "v": x["v_out"]}
    if x["op"] == "attend":
        R.paged_q4_attention(sh, x["q"], x["k_codes"], x["k_scales"], x["v_codes"], x["v_scales"], x["table"], x["cu"], x["kv_lens"],
                             x["scale"], x["o"], x["lse"], x["workspace"])
        return {"o": x["o"], "lse": x["lse"]}
    if x["op"] == "release":
        R.paged_release(sh, x["first"], x["end"], x["table"], x["holders"], x["free"], x["free_state"], x["table_out"],
                        x["holders_out"], x["free_out"], x["workspace"])
        return _told(x, "holders_out", "free", "free_out")
    if x["op"] == "fork":
        R.paged_fork(sh, x["parents"], x["children"], x["table"], x["lens"], x["holders"], x["free"], x["free_state"], x["table_out"],
                     x["lens_out"], x["holders_out"], x["moves"], x["free_out"])
    else:
        R.paged_compact(sh, x["lens"], x["table"], x["holders"], x["table_out"], x["holders_out"], x["free"], x["free_out"], x["moves"],
                        x["workspace"])
    R.paged_copy(sh, x["moves"], *x["caches"])
    return _told(x, *(("table_out", "lens_out", "holders_out", "moves", "free_out", "caches") if x["op"] == "fork" else
                      ("table_out", "holders_out", "free", "moves", "free_out", "caches")))


def _told(x, *names):
    return {n: x[n] for n in names}


def _write(x):
    P, s = x["k_codes"].shape[:2]
    keep = x["slots"] >= 0
    to = torch.where(keep, x["slots"], torch.zeros_like(x["slots"]))
    T = to.numel()
    # the token that fills each slot (one place more, for tokens without a slot), then a choice slot by slot
    at = torch.where(keep, x["slots"], torch.full_like(x["slots"], P * s))
    by = torch.full((P * s + 1,), -1, dtype=torch.int64, device=at.device).scatter(0, at, torch.arange(T, device=at.device))[:-1]
    by = by.view(P, s, 1, 1)
    out = {}
    for n in "kv":
        for name, new in zip(("_codes", "_scales"), _quantise(x[n].float())):
            held = x[n + name].view(torch.uint8)
            held.copy_(torch.where(by >= 0, new.view(torch.uint8)[by.clamp(min=0)[..., 0, 0]], held))
        got = _values(x[n + "_codes"][to // s, to % s], x[n + "_scales"].view(torch.uint8)[to // s, to % s].view(torch.float8_e4m3fn))
        x[n + "_out"].copy_(torch.where(keep[:, None, None], got, torch.zeros_like(got)))
        out[n] = x[n + "_out"]
    return out


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

    def held(n):
        codes = x[n + "_codes"][page, j % s].permute(0, 2, 1, 3)
        scales = x[n + "_scales"].view(torch.uint8)[page, j % s].permute(0, 2, 1, 3).contiguous().view(torch.float8_e4m3fn)
        table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=dev)
        pairs = torch.stack([table.repeat(16), table.repeat_interleave(16)], -1)  # a byte's two values
        return (pairs[codes.int()].view(N, Hkv, Tk, -1, 16) * scales.float()[..., None]).view(N, Hkv, Tk, D)

    pos = (kv - new)[:, None] + i
    seen = (j <= pos[..., None]) & (i < new[:, None])[..., None]
    if x["window"]:
        seen &= j > pos[..., None] - x["window"]
    logits = torch.matmul(q, held("k").transpose(-1, -2)).mul_(x["scale"]).view(N, Hkv, g, Tq, Tk)
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    weights = logits.sub_(top).exp_()
    total = weights.sum(-1, keepdim=True)
    o = torch.matmul(weights.view(N, Hkv, g * Tq, Tk), held("v")).view(N, Hkv, g, Tq, D)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log())[..., 0]
    # back to one row a token
    t = torch.arange(x["T"], device=dev)
    n = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[n]
    o = o.permute(0, 3, 1, 2, 4).reshape(N, Tq, Hq, D)[n, at].to(x["q"].dtype)
    lse = lse.permute(0, 3, 1, 2).reshape(N, Tq, Hq)[n, at].contiguous()
    return {"o": o, "lse": lse}


def _counts(pages, P):
    """How often each page is there; numbers outside the pool are passed over."""
    at = torch.where((pages >= 0) & (pages < P), pages, torch.full_like(pages, P)).long().flatten()
    return torch.zeros(P + 1, dtype=torch.int32, device=pages.device).scatter_add(0, at, torch.ones_like(at, dtype=torch.int32))[:P]


def _copy(x):
    """Pages moves[:, 0] to moves[:, 1], page by page chosen: the page that goes to each place, or its own."""
    P = x["P"]
    own_id = torch.arange(P + 1, device=x["moves"].device)
    m = x["moves"].long()
    to = torch.where(m[:, 1] >= 0, m[:, 1], torch.full_like(m[:, 1], P))
    by = own_id.scatter(0, to, m[:, 0])[:P]
    moved = by != own_id[:P]
    for c in x["caches"]:
        c.copy_(torch.where(moved.view(P, 1, 1, 1), c[by.clamp(min=0)], c))


def _fork(x):
    s, P, width = x["page"], x["P"], x["width"]
    src, dst = x["parents"].long(), x["children"].long()
    head, count = x["free_state"][0].long(), x["free_state"][1].long()
    L = x["lens"][src].long()
    full = L // s
    part = L % s > 0
    at = part.cumsum(0) - part.long()
    fresh = x["free"][((head + at) % P).clamp(min=0)]
    fresh = torch.where(part & (at < count), fresh, torch.full_like(fresh, -1))
    col = torch.arange(width, device=src.device)[None, :]
    rows = x["table"][src]
    shared = col < full[:, None]
    last = rows.gather(1, full.clamp(max=width - 1)[:, None])[:, 0]
    out = torch.where(shared, rows, torch.where((col == full[:, None]) & part[:, None], fresh[:, None], x["table_out"][dst]))
    x["table_out"].index_copy_(0, dst, out)
    x["lens_out"].index_copy_(0, dst, x["lens"][src])
    x["holders_out"].copy_(x["holders"] + _counts(torch.where(shared, rows, torch.full_like(rows, -1)), P))
    there = fresh >= 0
    x["moves"].copy_(torch.where(there[:, None], torch.stack([last, fresh], -1), torch.full_like(x["moves"], -1)))
    wanted = part.long().sum()
    taken = torch.minimum(wanted, count)
    x["free_out"].copy_(torch.stack([(head + taken) % P, count - taken, wanted - taken]))
    _copy(x)
    return _told(x, "table_out", "lens_out", "holders_out", "moves", "free_out", "caches")


def _release(x):
    P, width = x["P"], x["width"]
    head, count = x["free_state"][0].long(), x["free_state"][1].long()
    col = torch.arange(width, device=head.device)[None, :]
    goes = (col >= x["first"][:, None]) & (col < x["end"][:, None])
    n = _counts(torch.where(goes, x["table"], torch.full_like(x["table"], -1)), P)
    freed = n > x["holders"]
    x["holders_out"].copy_((x["holders"] - n).clamp(min=0))
    place = (head + count + freed.cumsum(0) - 1) % P
    ring = torch.cat([x["free"], x["free"][:1]])
    ring.scatter_(0, torch.where(freed, place, torch.full_like(place, P)), torch.arange(P, dtype=torch.int32, device=head.device))
    x["free"].copy_(ring[:P])
    x["free_out"].copy_(torch.stack([head, count + freed.sum(), torch.zeros_like(head)]))
    return _told(x, "holders_out", "free", "free_out")


def _compact(x):
    s, P, width = x["page"], x["P"], x["width"]
    col = torch.arange(width, device=x["lens"].device)[None, :]
    live = col < ((x["lens"].long() + s - 1) // s)[:, None]
    used = _counts(torch.where(live, x["table"], torch.full_like(x["table"], -1)), P) > 0
    U = used.sum()
    p = torch.arange(P, device=U.device)
    above, hole = used & (p >= U), ~used & (p < U)
    most = P // 2
    far, spare = torch.full_like(p, most), torch.full((most + 1,), -1, dtype=torch.int64, device=U.device)
    up, down = above.cumsum(0) - 1, hole.cumsum(0) - 1  # which of those it is, in ascending order
    src = spare.scatter(0, torch.where(above, up, far), torch.where(above, p, -torch.ones_like(p)))[:most]
    dst = spare.scatter(0, torch.where(hole, down, far), torch.where(hole, p, -torch.ones_like(p)))[:most]
    x["moves"].copy_(torch.stack([src, dst], -1))
    to = torch.where(above, dst[up.clamp(min=0, max=max(0, most - 1))], p) if most else p
    x["table_out"].copy_(torch.where(live, to[x["table"].long().clamp(0, P - 1)].int(), x["table"]))
    held = torch.zeros(P + 1, dtype=torch.int32, device=U.device)
    x["holders_out"].copy_(held.scatter(0, torch.where(used, to, torch.full_like(to, P)), x["holders"])[:P])
    x["free"].copy_(torch.where(p < P - U, p + U, x["free"]))
    zero = torch.zeros_like(U)
    x["free_out"].copy_(torch.stack([zero, P - U, zero]))
    _copy(x)
    return _told(x, "table_out", "holders_out", "free", "moves", "free_out", "caches")


# ------------------------------------------------------------------------------------------------ in 64 bits
def _e4m3():
    """The finite values of E4M3 from 2^-9 on, ascending: a fraction of 3 bits, subnormal below 2^-6, the last one 448."""
    v = [m * 2.0 ** -9 for m in range(1, 8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64, device="cuda")


def _nearest(x, grid):
    """The place in an ascending grid of the value nearest to x >= 0, of two as near the even place (places count from grid[0])."""
    mid = (grid[1:] + grid[:-1]) / 2
    low, high = torch.searchsorted(mid, x, right=False), torch.searchsorted(mid, x, right=True)
    return torch.where(low % 2 == 0, low, high)


def exact(case, seed):
    if case["op"] == "release":
        return None  # whole numbers alone
    x = prepare(case, seed)
    grid = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
    if case["op"] == "write":
        out = {}
        for n in "kv":
            v = x[n].double().unflatten(-1, (-1, 16))
            top = v.abs().amax(-1, keepdim=True)
            e = torch.cat([torch.zeros(1, dtype=torch.float64, device="cuda"), _e4m3()])
            s = e[_nearest(top / 6, e).clamp(min=1)]
            y = torch.copysign(grid[_nearest(v.abs() / s, grid)], v) * s
            y = torch.where(torch.isfinite(top), y, torch.full_like(y, math.nan)).flatten(-2)
            out[n] = torch.where((x["slots"] >= 0)[:, None, None], y, torch.zeros_like(y))
        return out
    if case["op"] != "attend":
        # what is moved, apart from the way it is found: children's last pages, and every used page in its new place
        s, lens = case["page"], _pages(case)[0]
        caches = [c.double() for c in x["caches"]]
        table = x["table"].long()
        if case["op"] == "fork":
            part = [i for i, n in enumerate(x["parents"].tolist()) if lens[n] % s]
            from_ = [int(table[n, lens[n] // s]) for n in (x["parents"].tolist()[i] for i in part)]
            head = int(x["free_state"][0])
            to = [int(x["free"][(head + i) % x["P"]]) for i in range(len(part))]
        else:
            used = sorted({p for n, m in enumerate(lens) for p in table[n, :-(-m // s)].tolist()})
            from_ = [p for p in used if p >= len(used)]
            to = sorted(set(range(len(used))) - set(used))
        if to:
            a, b = (torch.tensor(v, device="cuda") for v in (from_, to))
            for c in caches:
                c[b] = c[a]
        return {"caches": caches}
    if work(case)["flops"] > 4e12:
        return None
    s, g, W = case["page"], case["Hq"] // case["Hkv"], case["window"]
    signed = torch.cat([grid, -grid])

    def held(n, at, j, h):
        codes = x[n + "_codes"][at, j % s, h].long()
        both = torch.stack([signed[codes & 15], signed[codes >> 4]], -1)
        scales = x[n + "_scales"].view(torch.uint8)[at, j % s, h].contiguous().view(torch.float8_e4m3fn).double()
        return both.flatten(-2) * scales.repeat_interleave(16, -1)

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
                Q = x["q"][first + a:first + b, h * g:(h + 1) * g].double().transpose(0, 1)
                S = (Q @ held("k", at, j, h).T * x["scale"]).masked_fill(hidden, -math.inf)
                Z = torch.logsumexp(S, -1)
                o[first + a:first + b, h * g:(h + 1) * g] = (torch.exp(S - Z[..., None]) @ held("v", at, j, h)).transpose(0, 1)
                lse[first + a:first + b, h * g:(h + 1) * g] = Z.T
        first += new
    return {"o": o, "lse": lse}


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    s = case["page"]
    if case["op"] in ("fork", "release", "compact"):
        lens, P = _pages(case)
        held = [-(-n // s) for n in lens]
        if case["op"] == "release":
            ended = sum(sorted(held)[:_ended(case)])  # (which ones end is the seed's)
            return {"bytes": 8 * case["N"] + 4 * ended + 8 * ended + 4 * P, "flops": 0}
        page = 2 * case["layers"] * s * case["Hkv"] * case["D"] * (2 if case["type"] == "bf16" else 4)
        if case["op"] == "fork":
            copies = sum(n % s > 0 for n in lens) * case["each"]
            shared = sum(n // s for n in lens)
            ids = 4 * shared + (4 * shared + 12) * case["each"] + 8 * P
        else:
            used = sum(held)
            copies = used - used * used // P  # of scattered pages, the share past the first `used`
            ids = 8 * used + 12 * P
        return {"bytes": 2 * copies * page + ids, "flops": 0}
    size = 2 if case["type"] == "bf16" else 4
    D, Hkv = case["D"], case["Hkv"]
    row = D // 2 + D // 16  # a token's codes and scales of one head
    if case["op"] == "write":
        return {"bytes": case["T"] * (8 + 2 * Hkv * (2 * D * size + 2 * row)), "flops": 0}
    W, Hq = case["window"], case["Hq"]
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
    return {"bytes": 2 * keys * Hkv * row + 2 * T * Hq * D * size + 4 * T * Hq, "flops": 4 * D * pairs * Hq}
