"""Properties of the kernel sources that no run shows reliably: they guard against orders of
execution that the hardware may take but hardly ever does."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_recurrent_rnn_gb300", "csrc")


def source(name):
    """The file without its comments."""
    s = open(os.path.join(CSRC, name)).read()
    s = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), s, flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


def kernels(name):
    """The bodies of the file's kernels."""
    out = []
    s = source(name)
    for m in re.finditer(r"__global__", s):
        i = s.index("{", s.index("(", m.end() + (re.match(r"\s*void\s+__launch_bounds__\([^{]*?\)\s*\n", s[m.end():]) or
                                                re.match("", "")).end()))
        depth, j = 0, i
        while True:
            depth += {"{": 1, "}": -1}.get(s[j], 0)
            j += 1
            if not depth:
                break
        out.append(s[i:j])
    return out


FILES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu")))


def early(body):
    """The kernel waits for the grid before it (programmatic stream serialisation)."""
    return "griddep_wait" in body


def test_kernels_are_found():
    assert sum(early(b) for f in FILES for b in kernels(f)) >= 6


@pytest.mark.parametrize("name", FILES)
def test_the_next_grid_starts_after_tmem_is_held(name):
    """A grid that waits for this one may hold TMEM meanwhile: were it let in before this grid's
    allocation, neither would go on.  So the warp that allocates gives the signal, or a CTA
    barrier lies between."""
    for body in kernels(name):
        if not early(body) or "tmem_alloc" not in body:
            continue
        alloc = re.search(r"if \(([^\n]*)\) \{\s*(?:tc::)?tmem_alloc", body)
        go = re.search(r"(?:if \(([^\n]*)\) )?(?:tc::)?griddep_launch_dependents\(\)", body)
        assert alloc and go and alloc.start() < go.start()
        assert go.group(1) == alloc.group(1) or "__syncthreads()" in body[alloc.end():go.start()], name


def loops(body):
    """The bodies of the innermost braced loops around each TMEM access."""
    spans = []
    for m in re.finditer(r"\bfor \(", body):
        depth, i = 0, m.end() - 1
        while True:
            depth += {"(": 1, ")": -1}.get(body[i], 0)
            i += 1
            if not depth:
                break
        while body[i] in " \n":
            i += 1
        if body[i] != "{":
            continue
        j, depth = i, 0
        while True:
            depth += {"{": 1, "}": -1}.get(body[j], 0)
            j += 1
            if not depth:
                break
        spans.append((i, j))
    for m in re.finditer(r"tc::tmem_(ld|st)\d", body):
        inside = [s for s in spans if s[0] < m.start() < s[1]]
        if inside:
            i, j = max(inside)
            yield body[i:j], m.start() - i


@pytest.mark.parametrize("name", ["paged_attn_tc.cu", "paged_attn_few.cu"])
def test_tmem_is_read_by_converged_warps(name):
    """tcgen05's loads and stores want all lanes of the warp there: a loop whose body branches by
    thread brings them together before the access."""
    seen = 0
    for body in kernels(name):
        for loop, at in loops(body):
            if re.search(r"\b(mine|tid)\b", loop):
                seen += 1
                assert re.search(r"__syncwarp\(\)|ctl\.wait\(|tf_any\(", loop[:at]), loop[:200]
    assert seen


@pytest.mark.parametrize("name", [f for f in FILES if f.startswith("paged")])
def test_aligned_cluster_barriers_are_met_by_converged_warps(name):
    for m in re.finditer(r"barrier\.cluster\.arrive[.\w]*\.aligned", source(name)):
        assert re.search(r"__syncwarp\(\);\s*asm volatile\(\"$", source(name)[:m.start()])


@pytest.mark.parametrize("name", sorted({f for f in FILES if any(early(b) for b in kernels(f))} | {"paged.cuh", "paged_tc.cuh"}))
def test_kernels_that_start_early_use_coherent_loads(name):
    """The non-coherent path is for memory that nothing writes while the kernel lives; the life of
    a kernel with programmatic stream serialisation overlaps that of the grid before it."""
    assert not re.search(r"__ldg\b|\.nc\b|ld\.global\.nc|__restrict__", source(name))
