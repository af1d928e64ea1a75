"""CPU checks of the paged-cache entry points (include/paged_attn.h): every declared symbol is
exported, scratch is sized, and wrong arguments are refused on the host before any CUDA call
(fake, never dereferenced addresses)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from linear_recurrent_rnn_gb300 import build as B_
from linear_recurrent_rnn_gb300 import librglru as R

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "paged_attn.h")
A = 1 << 20


@pytest.fixture(scope="module")
def lib():
    B_.build()
    return R.lib()


def P(v):
    return None if v is None else ctypes.c_void_p(v)


def shape(**kw):
    d = dict(num_seqs=2, tokens=3, Hq=4, Hkv=2, D=64, num_pages=8, page_size=16, table_width=4)
    d.update(kw)
    return R.make_paged_shape(**d)


def test_declared_symbols_are_exported(lib):
    src = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(paged_[a-z_]+)\s*\(", src))
    assert names == set(R.EXPORTS_PAGED)
    out = subprocess.run(["nm", "-D", "--defined-only", B_.LIB], capture_output=True, text=True,
                         check=True).stdout
    assert names <= set(re.findall(r"\bT (paged_\w+)", out))


BAD_CACHE = [
    (dict(num_seqs=0), R.ERR_INVALID_ARG), (dict(tokens=-1), R.ERR_INVALID_ARG),
    (dict(num_pages=0), R.ERR_INVALID_ARG), (dict(table_width=0), R.ERR_INVALID_ARG),
    (dict(page_size=0), R.ERR_INVALID_ARG), (dict(page_size=24), R.ERR_UNSUPPORTED),
    (dict(page_size=4), R.ERR_UNSUPPORTED), (dict(page_size=8192), R.ERR_UNSUPPORTED),
    (dict(num_seqs=8193), R.ERR_UNSUPPORTED),
    (dict(num_pages=1 << 20, page_size=4096), R.ERR_UNSUPPORTED),
]
BAD_HEADS = [
    (dict(Hkv=0), R.ERR_INVALID_ARG), (dict(D=0), R.ERR_INVALID_ARG), (dict(io=7), R.ERR_INVALID_ARG),
    (dict(D=4), R.ERR_UNSUPPORTED), (dict(D=264), R.ERR_UNSUPPORTED), (dict(D=68), R.ERR_UNSUPPORTED),
]
BAD_QUERIES = [
    (dict(Hq=0), R.ERR_INVALID_ARG), (dict(Hq=3), R.ERR_INVALID_ARG), (dict(window=-1), R.ERR_INVALID_ARG),
    (dict(Hq=130, Hkv=2), R.ERR_UNSUPPORTED),
]


def plan(lib, sh, **kw):
    a = {n: A for n in ("cached", "new", "ring", "state", "table", "cu", "kv", "pos", "slots", "out")}
    a.update(kw)
    return lib.paged_plan(ctypes.byref(sh), *[P(a[n]) for n in (
        "cached", "new", "ring", "state", "table", "cu", "kv", "pos", "slots", "out")], None)


def write(lib, sh, strides=None, **kw):
    a = {n: A for n in ("k", "v", "slots", "kc", "vc")}
    a.update(kw)
    return lib.paged_kv_write(ctypes.byref(sh), strides, *[P(a[n]) for n in ("k", "v", "slots", "kc", "vc")], None)


def attend(lib, sh, strides=None, scale=0.1, **kw):
    a = {n: A for n in ("q", "kc", "vc", "table", "cu", "kv", "o", "lse", "ws")}
    a.update(kw)
    return lib.paged_attention(ctypes.byref(sh), strides, *[P(a[n]) for n in ("q", "kc", "vc", "table", "cu", "kv")],
                               scale, P(a["o"]), P(a["lse"]), P(a["ws"]), None)


@pytest.mark.parametrize("kw,want", BAD_CACHE)
def test_cache_sizes_are_refused(lib, kw, want):
    for f in (plan, write, attend):
        assert f(lib, shape(**kw)) == want
    assert R.paged_attention_workspace_bytes(shape(**kw)) == 0


@pytest.mark.parametrize("kw,want", BAD_HEADS)
def test_head_sizes_are_refused(lib, kw, want):
    for f in (write, attend):
        assert f(lib, shape(**kw)) == want
    assert R.paged_attention_workspace_bytes(shape(**kw)) == 0


@pytest.mark.parametrize("kw,want", BAD_QUERIES)
def test_query_sizes_are_refused(lib, kw, want):
    assert attend(lib, shape(**kw)) == want
    assert R.paged_attention_workspace_bytes(shape(**kw)) == 0


def test_pointers_are_refused(lib):
    for n in ("cached", "new", "ring", "state", "table", "cu", "kv", "pos", "slots", "out"):
        assert plan(lib, shape(), **{n: None}) == R.ERR_INVALID_ARG
        assert plan(lib, shape(), **{n: A + 2}) == R.ERR_INVALID_ARG
    for n in ("k", "v", "slots", "kc", "vc"):
        assert write(lib, shape(), **{n: None}) == R.ERR_INVALID_ARG
        assert write(lib, shape(), **{n: A + 4}) == R.ERR_INVALID_ARG
    for n in ("q", "kc", "vc", "table", "cu", "kv", "o", "ws"):
        assert attend(lib, shape(), **{n: None}) == R.ERR_INVALID_ARG
        assert attend(lib, shape(), **{n: A + 2}) == R.ERR_INVALID_ARG
    assert attend(lib, shape(), lse=A + 2) == R.ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [0.0, -1.0, float("inf"), float("nan")])
def test_scales_are_refused(lib, scale):
    assert attend(lib, shape(), scale=scale) == R.ERR_INVALID_ARG


def test_strides_are_refused(lib):
    names = [n for n, _ in R.PagedStrides._fields_]
    good = {n: 64 for n in names}
    for bad in (0, -64, 4):   # 4 bf16: 8 bytes
        for n in names:
            st = R.PagedStrides(**dict(good, **{n: bad}))
            if n[0] not in "qo":
                assert write(lib, shape(), st) == R.ERR_UNSUPPORTED
            if n[:2] not in ("k_", "v_"):
                assert attend(lib, shape(), st) == R.ERR_UNSUPPORTED


def test_no_tokens_is_no_work(lib):
    """Nothing is read, written or launched."""
    assert write(lib, shape(tokens=0), k=None, v=None, slots=None, kc=None, vc=None) == R.OK
    assert attend(lib, shape(tokens=0), q=None, kc=None, vc=None, o=None, ws=None) == R.OK


def test_workspace_is_sized(lib):
    for io in (R.F32, R.BF16):
        small = R.paged_attention_workspace_bytes(shape(io=io, D=64))
        large = R.paged_attention_workspace_bytes(shape(io=io, D=256))
        assert 0 < small < large < 256 << 20


def test_binding_refuses_wrong_tensors(lib):
    sh = shape()
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):   # not on a GPU
        R.paged_kv_write(sh, q[:, :2], q[:, :2], torch.zeros(3, dtype=torch.int64), q, q)
    with pytest.raises(ValueError):   # another shape
        R.paged_attention(sh, q[:2], q, q, q, q, q, 1.0, q, None, q)
    with pytest.raises(ValueError):   # another type
        R.paged_attention(sh, q.float(), q, q, q, q, q, 1.0, q, None, q)
