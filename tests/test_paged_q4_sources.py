"""Properties of the sources of the 4-bit cache's attention that no run shows reliably."""
import itertools
import re

import pytest

from test_kernel_sources import kernels, source


def value(expr, names):
    """A constant expression of C++ with ternaries, in whole numbers."""
    depth = 0
    for i, ch in enumerate(expr):
        depth += {"(": 1, ")": -1}.get(ch, 0)
        if ch == "?" and depth == 0:
            nested, j, level = 0, i + 1, 0
            while nested or level or expr[j] != ":":
                level += {"(": 1, ")": -1}.get(expr[j], 0)
                nested += (expr[j] == "?") - (expr[j] == ":")
                j += 1
            return value(expr[i + 1:j] if value(expr[:i], names) else expr[j + 1:], names)
    expr = expr.replace("C::", "").replace("||", " or ").replace("&&", " and ").replace("/", "//")
    return eval(expr.strip(), {"__builtins__": {}}, dict(names))


def constants(struct, names):
    """The struct's whole-number constants, for these template arguments, as far as they can be worked out."""
    out = dict(names)
    for name, expr in re.findall(r"static constexpr (?:int|uint32_t) (\w+) = ([^;]+);", struct):
        for n, e in re.findall(r"(\w+) = ([^,;]+(?:\([^)]*\))?[^,;]*)", f"{name} = {expr}"):
            try:
                out[n] = value(e, out)
            except (NameError, SyntaxError):
                pass
    return out


# widths, rows of a tile, float32: the instances that a call reaches
INSTANCES = ([(d, r, False) for d, r in itertools.product((64, 128, 256), (4, 8, 16))] + [(256, 32, False)]
             + [(d, r, True) for d, r in itertools.product((64, 128, 256), (8, 16))])


def test_the_evaluator():
    assert [value("R == 32 ? 1 : R == 16 || DP == 256 ? 2 : 4", dict(R=r, DP=d)) for r, d in ((32, 256), (16, 64), (4, 256), (4, 64))] == [1, 2, 2, 4]
    assert value("(3 * K + 15) / 16 * 16", dict(K=6)) == 32


@pytest.mark.parametrize("DP,R,F32", INSTANCES)
def test_scores_fit_the_array_that_they_are_read_into(DP, R, F32):
    """A read from TMEM fills 16 elements whether the step has as many scores or not."""
    s = source("paged_attn_q4.cu")
    c = constants(s[s.index("struct Tq {"):s.index("template <int DP, int R, bool F32>\n__global__")], dict(DP=DP, R_=R, R=R, F32_=F32, F32=F32))
    body, = kernels("paged_attn_q4.cu")
    m = re.search(r"float x\[([^\]]+)\];\s*#pragma unroll\s*for \(int c = 0; c < ([^;]+); c \+= 16\)\s*tc::tmem_ld16\([^;]*\(x \+ c\)\);", body)
    size, end = value(m.group(1), c), value(m.group(2), c)
    assert end >= c["KT"] * c["COLS"]
    assert all(at + 16 <= size for at in range(0, end, 16))


def test_sums_are_written_once_every_warp_has_read_the_maxima():
    """s_red holds the warps' maxima of a step, then their sums.  All threads read the maxima behind a barrier; a warp may
    be done with its weights while another still reads, so between the weights' arrival and the sums' store
    lies what waits for all four warps: the products of those weights, or a barrier."""
    body, = kernels("paged_attn_q4.cu")
    handed_in = body.index("tc::mbar_arrive(&p_full[b])")
    store = body.index("s_red[warp]", handed_in)
    assert re.search(r"ctl\.wait\(&pv_done\[\(step - 1\) & 1\]|tf_any\(|__syncthreads\(", body[handed_in:store])
    read = body.index("row_sum(", store)
    assert re.search(r"tf_any\(|__syncthreads\(", body[store:read])


def test_every_item_begins_with_a_barrier_of_the_softmax_warps():
    """Maxima, references and factors in shared memory are read up to the end of an item, and written from its first
    step on."""
    body, = kernels("paged_attn_q4.cu")
    start = body.index("ctl.wait(&i_full[ni % TA_ITEMS]")
    assert "tf_any(!ok)" in body[start:body.index("s_ref[", start)]
