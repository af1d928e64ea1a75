"""Builds librglru.so in-tree with nvcc for sm_103a (GB300), and the Python module beside it.

Each translation unit is compiled in parallel; the CUDA runtime is linked statically and the
driver API is reached at run time through cudaGetDriverEntryPoint, so the library loads on a
machine without a GPU (where only its symbols can be inspected).  The module (csrc/binding.cpp:
checks of tensors and the calls of the paged cache) is compiled against the installed torch and
Python; it does not link the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "librglru.so")


def binding_path() -> str:
    """The Python module's file.  It reads torch's tensors through the headers that it was compiled
    with, so its name says which torch and which Python those are: another's is not there, rather
    than loaded."""
    try:
        import torch
        version = torch.__version__
    except ImportError:
        version = "-none"
    return os.path.join(BUILD, f"rglru_binding-torch{version}-{sysconfig.get_config_var('SOABI')}.so")


BINDING = binding_path()
SOURCES = ["api.cu", "scan_simt.cu", "gemm_simt.cu", "noalloc.cu", "host_util.cu", "fused_fwd.cu", "fused_bwd.cu",
           "decode.cu", "varlen.cu", "delta_rule.cu", "proj_tc.cu", "paged.cu", "paged_attn_simt.cu",
           "paged_attn_tc.cu", "paged_attn_few.cu"]
HEADERS = ["common.cuh", "internal.h", "tc.cuh", "host_util.h", "lookback.cuh",
           "paged.cuh", "paged_tc.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "librglru.h"))
    files.append(os.path.join(ROOT, "include", "delta_rule.h"))
    files.append(os.path.join(ROOT, "include", "paged_attn.h"))
    files.append(os.path.join(CSRC, "binding.cpp"))
    files.append(os.path.abspath(__file__))
    return files


def missing_headers() -> list:
    """Headers that the Python module wants and that are not installed; the library wants none of them."""
    want = [os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    try:
        import torch
        want.append(os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd",
                                 "python_variable.h"))
    except ImportError:
        want.append("torch/csrc/autograd/python_variable.h")
    return [f for f in want if not os.path.exists(f)]


def stale() -> bool:
    made = [LIB] if missing_headers() else [LIB, BINDING]
    if not all(map(os.path.exists, made)):
        return True
    t = min(map(os.path.getmtime, made))
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every kernel translation unit and link librglru.so, compile the Python module (without
    its headers: a note instead, and the calls that need the module raise); returns the library's path."""
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        tmp = obj + f".tmp{os.getpid()}.o"  # (whole for another process that builds meanwhile)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", tmp]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        os.replace(tmp, obj)
        return obj

    def compile_binding():
        import torch
        root = os.path.dirname(torch.__file__)
        tmp = BINDING + f".tmp{os.getpid()}"
        cmd = [nvcc, "-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", os.path.join(CSRC, "binding.cpp"),
               "-o", tmp, "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
               "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        missing = missing_headers()
        module = None if missing else ex.submit(compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)  # (there whatever becomes of the module)
        if module:
            module.result()
        else:
            sys.stderr.write(f"librglru: the Python module is not built: {', '.join(missing)} missing\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
