"""Builds the SFA CUDA library in-tree: kv_cache_compression_sfa_b200/libsfa.so
(and _fast.so beside it, where the host has a C++ compiler and the headers).

nvcc compiles every ``csrc/*.cu`` for sm_100a (B200) only and links them into
one shared library exposing the C ABI of ``include/sfa.h``.  Runs without a
GPU (cross-compilation).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsfa.so")
FAST_SRC = os.path.join(CSRC, "binding_fast.cpp")
FAST_LIB = os.path.join(PKG, "_fast.so")
BUILD_DIR = os.path.join(PKG, "_build")
FAST_STAMP = os.path.join(BUILD_DIR, "_fast.built_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "sfa.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if up_to_date() and not force and not ptxas_info:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    return LIB


def fast_stamp() -> str:
    """What the extension was built for: another torch or Python has other
    objects behind the same names."""
    import torch
    return f"torch {torch.__version__}, Python {sys.version_info.major}.{sys.version_info.minor}"


def build_fast(force: bool = False, verbose: bool = False):
    """The Python extension of the per-step paged cache calls, against torch's
    headers (host code only).  The binding works without it, slower: where it
    cannot be built, a warning says why and the result is None."""
    deps = (FAST_SRC, os.path.join(INCLUDE, "sfa.h"), os.path.abspath(__file__))
    stamp = fast_stamp()
    if (not force and os.path.exists(FAST_LIB) and os.path.exists(FAST_STAMP) and
            open(FAST_STAMP).read() == stamp and
            all(os.path.getmtime(d) <= os.path.getmtime(FAST_LIB) for d in deps)):
        return FAST_LIB
    import sysconfig

    import torch
    tmp = FAST_LIB + f".tmp{os.getpid()}"
    try:
        from torch.utils import cpp_extension
        inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], INCLUDE,
                                               os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DSFA_BUILT_FOR="{stamp}"',
               *[f"-isystem{d}" for d in inc], FAST_SRC, "-o", tmp,
               # torch's own libraries, loaded by the time the module is
               *[f"-L{d}" for d in cpp_extension.library_paths()],
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    except (OSError, RuntimeError, ImportError, subprocess.CalledProcessError) as e:
        if os.path.exists(FAST_LIB):
            os.remove(FAST_LIB)  # of other sources, or of another torch
        warnings.warn(f"{os.path.basename(FAST_LIB)} was not built, paged cache calls go through ctypes: {e}")
        return None
    os.replace(tmp, FAST_LIB)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(FAST_STAMP, "w") as f:
        f.write(stamp)
    return FAST_LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    build_fast(force="--force" in sys.argv, verbose=True)
    print(LIB)
