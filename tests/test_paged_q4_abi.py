"""CPU checks of the cache in 4 bits (include/paged_q4.h): symbols, scratch, refusals on the host before any
CUDA call (fake, never dereferenced addresses), and its oracle."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from linear_recurrent_rnn_gb300 import build as B_
from linear_recurrent_rnn_gb300 import librglru as R
from oracle import paged_q4 as O
from test_paged_abi import A, BAD_CACHE, BAD_QUERIES, P, lib, shape  # noqa: F401  (lib: a fixture)

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "paged_q4.h")
CACHE = ("kc", "ks", "vc", "vs")
BAD_HEADS = [
    (dict(Hkv=0), R.ERR_INVALID_ARG), (dict(D=0), R.ERR_INVALID_ARG), (dict(io=7), R.ERR_INVALID_ARG),
    (dict(D=8), R.ERR_UNSUPPORTED), (dict(D=272), R.ERR_UNSUPPORTED), (dict(D=72), R.ERR_UNSUPPORTED),
    (dict(D=65), R.ERR_UNSUPPORTED),
]
SIZES = BAD_CACHE + [(dict(tokens=2 ** 30 + 1), R.ERR_UNSUPPORTED), (dict(num_seqs=8192, table_width=2 ** 18), R.ERR_UNSUPPORTED)]


def call(f, names, sh, strides=None, scale=None, **kw):
    a = dict({n: A for n in names}, **kw)
    v = [P(a[n]) for n in names]
    if scale is not None:
        v.insert(names.index("o"), scale)
    return f(ctypes.byref(sh), strides, *v, None)


def write(lib, sh, strides=None, **kw):  # noqa: F811
    return call(lib.paged_q4_write, ("k", "v", "slots") + CACHE, sh, strides, **kw)


def read(lib, sh, strides=None, **kw):  # noqa: F811
    return call(lib.paged_q4_read, ("slots",) + CACHE + ("k", "v"), sh, strides, **kw)


def attend(lib, sh, strides=None, scale=0.1, **kw):  # noqa: F811
    return call(lib.paged_q4_attention, ("q",) + CACHE + ("table", "cu", "kv", "o", "lse", "ws"), sh, strides, scale, **kw)


def test_declared_symbols_are_exported(lib):  # noqa: F811
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(paged_q4_[a-z_]+)\s*\(", src))
    assert names == set(R.EXPORTS_Q4)
    out = subprocess.run(["nm", "-D", "--defined-only", B_.LIB], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r"\bT (paged_\w+)", out))
    fields = re.search(r"typedef struct \{(.*?)\} paged_q4_strides;", src, re.S).group(1)
    assert re.findall(r"\w+(?=[,;])", fields) == [n for n, _ in R.PagedQ4Strides._fields_]


@pytest.mark.parametrize("kw,want", SIZES + BAD_HEADS)
def test_sizes_are_refused(lib, kw, want):  # noqa: F811
    for f in (write, read, attend):
        assert f(lib, shape(**kw)) == want
    assert R.paged_q4_attention_workspace_bytes(shape(**kw)) == 0


@pytest.mark.parametrize("kw,want", BAD_QUERIES)
def test_query_sizes_are_refused(lib, kw, want):  # noqa: F811
    assert attend(lib, shape(**kw)) == want
    assert R.paged_q4_attention_workspace_bytes(shape(**kw)) == 0


def test_pointers_are_refused(lib):  # noqa: F811
    for f in (write, read, attend):
        for n in CACHE + (("q", "table", "cu", "kv", "o", "ws") if f is attend else ("k", "v", "slots")):
            assert f(lib, shape(), **{n: None}) == R.ERR_INVALID_ARG, n
            assert f(lib, shape(), **{n: A + 2}) == R.ERR_INVALID_ARG, n
        for n in ("kc", "vc"):
            assert f(lib, shape(), **{n: A + 8}) == R.ERR_INVALID_ARG, n
    assert attend(lib, shape(), lse=A + 2) == R.ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan"), 2.4e38])
def test_scales_are_refused(lib, scale):  # noqa: F811
    assert attend(lib, shape(), scale=scale) == R.ERR_INVALID_ARG


def test_strides_are_refused(lib):  # noqa: F811
    good = {n: 64 for n, _ in R.PagedQ4Strides._fields_}
    for n in good:
        # 4 bf16 are 8 bytes, 8 bytes of codes no whole 16, 2 of scales no whole 4
        for bad in (0, -64, 8 if n[1:3] == "c_" else 2 if n[1:3] == "s_" else 4):
            st = R.PagedQ4Strides(**dict(good, **{n: bad}))
            cache = n[1:3] in ("c_", "s_")
            if cache or n[0] in "qo":
                assert attend(lib, shape(), st) == R.ERR_UNSUPPORTED
            if cache or n[0] in "kv":
                assert write(lib, shape(), st) == R.ERR_UNSUPPORTED
                assert read(lib, shape(), st) == R.ERR_UNSUPPORTED


def test_no_tokens_is_no_work(lib):  # noqa: F811
    assert write(lib, shape(tokens=0), k=None, v=None, slots=None, kc=None) == R.OK
    assert read(lib, shape(tokens=0), k=None, v=None, slots=None, ks=None) == R.OK
    assert attend(lib, shape(tokens=0), q=None, kc=None, o=None, ws=None) == R.OK


def test_workspace_is_sized(lib):  # noqa: F811
    for io in (R.F32, R.BF16):
        small, large = (R.paged_q4_attention_workspace_bytes(shape(io=io, D=D)) for D in (64, 256))
        assert 0 < small < large < 256 << 20


def test_binding_refuses_wrong_tensors(lib):  # noqa: F811
    sh = shape()
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    c = R.alloc_paged_q4_cache(sh, device="cpu")
    assert [tuple(t.shape) for t in c] == [(8, 16, 2, 32), (8, 16, 2, 4)] * 2
    with pytest.raises(ValueError, match="^k: "):   # not on a GPU
        R.paged_q4_write(sh, k, k, torch.zeros(3, dtype=torch.int64), *c)
    with pytest.raises(ValueError, match="^slots: "):
        R.paged_q4_read(sh, torch.zeros(3, dtype=torch.int64), *c, k, k)
    with pytest.raises(ValueError, match="^q: "):
        R.paged_q4_attention(sh, k, *c, k, k, k, 0.1, k, None, k)


# ---------------------------------------------------------------- the oracle
def test_oracle_tables():
    assert np.array_equal(torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), O.E4M3)
    assert np.all(np.diff(O.E4M3) > 0) and O.E4M3[-1] == 448


def test_oracle_keeps_what_it_can_hold():
    """Numbers that are a code times a scale, with a 6 among them, come back as they were."""
    for sc in (1, 8, 56, 100, 126):
        x = np.concatenate([O.E2M1, -O.E2M1]) * O.E4M3[sc]
        codes, scale = O.group(x)
        assert scale == sc
        assert np.array_equal(O.values(codes[0::2] | codes[1::2] << 4, np.array([scale], np.uint8)), x)


def test_oracle_errors_are_bounded():
    """At most (1 + 1/16) a / 6 off: half the widest gap, 1, times a scale that is at most 1/16 above a / 6; and
    where it is below, a / s is at most 6 (1 + 1/16), cut off at 6: less."""
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 32)) * np.exp(rng.standard_normal((40, 1)) * 2)
    y = O.values(*O.quantise(x)).reshape(40, 2, 16)
    x = x.reshape(40, 2, 16)
    assert np.all(np.abs(x - y) <= np.abs(x).max(-1, keepdims=True) / 6 * (1 + 1 / 16))
