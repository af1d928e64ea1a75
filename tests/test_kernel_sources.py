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
