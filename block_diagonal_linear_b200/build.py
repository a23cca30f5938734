"""Build libmonarch.so in-tree with nvcc for sm_100a, and then _mx4_native.so, the native half of the MX4
binding, with g++ against the installed torch.  The C ABI needs the first alone: where torch, its CUDA
libraries, Python's headers or a C++ compiler are missing, the second is left out with a warning, and the MX4
binding says so at its first use.

Usage: python -m block_diagonal_linear_b200.build  (or call build()).
"""
from __future__ import annotations

import os
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmonarch.so")
SOURCES = ["api.cu", "generic.cu", "tc_fwd.cu", "tc_rows.cu", "tc_wide.cu", "tc_split.cu", "tc_stage.cu", "tc_gemm.cu", "tc_pair.cu",
           "bwd_fast.cu", "bwd_gemm.cu", "linear.cu", "project.cu", "dyad.cu", "lattice.cu", "noalloc.cu",
           "mx4.cu", "mx4_quant.cu", "mx4_gemm.cu", "mx4_tc.cu", "mx4_rows.cu"]
NATIVE_LIB = os.path.join(PKG, "_mx4_native.so")
NATIVE_SOURCE = os.path.join(CSRC, "mx4_native.cpp")
HEADERS = ["common.cuh", "ptx.cuh", "tc_common.cuh", "tc_gemm.cuh", "mx4.cuh"]

NVCC_FLAGS = [
    "-O3",
    "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [*sources, os.path.join(ROOT, "include", "monarch.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def native_key(torch) -> str:
    """What _mx4_native.so is built for: it reads torch's C++ objects through this version's headers."""
    return "mx4 native: torch %s, cxx11 abi %d, %s" % (torch.__version__, torch.compiled_with_cxx11_abi(), sys.implementation.cache_tag)


def _native_stale(torch) -> bool:
    if _stale(NATIVE_LIB, [NATIVE_SOURCE]):
        return True
    with open(NATIVE_LIB, "rb") as f:
        return native_key(torch).encode() + b"\0" not in f.read()


def _build_native(torch, verbose: bool):
    import sysconfig

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    include = [os.path.join(base, "include"), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = NATIVE_LIB + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(), '-DMX4_NATIVE_KEY="%s"' % native_key(torch), *(a for p in include for a in ("-isystem", p)),
           NATIVE_SOURCE, "-o", tmp, "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, NATIVE_LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    _build_lib(force, verbose)
    try:
        import torch
        if force or _native_stale(torch):
            _build_native(torch, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        if os.path.exists(NATIVE_LIB) and _stale(NATIVE_LIB, [NATIVE_SOURCE]):
            os.remove(NATIVE_LIB)  # of older sources: it must not be taken for theirs
        warnings.warn("_mx4_native.so was not built (%s): the MX4 operators are left to the C entry points" % e)
    return LIB


def _build_lib(force: bool, verbose: bool) -> str:
    if not force and not _stale(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS]):
        return LIB
    objs = []
    bdir = os.path.join(PKG, "_build")
    os.makedirs(bdir, exist_ok=True)
    for src in SOURCES:
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + ".tmp%d" % os.getpid()
    subprocess.check_call([_nvcc(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                           *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
