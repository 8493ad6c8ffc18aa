"""Compile libkda.so in-tree with nvcc for sm_103a.

One translation unit per .cu file, compiled in parallel, then linked into a
shared library with the CUDA runtime linked statically (the library needs no
libcuda at load time; driver entry points are looked up at run time).  Beside it,
the marshalling of the full-attention layer's calls, compiled against the torch in use.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda.so")
    return path


def _compile(src: str, extra: list, build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, "-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC",
           "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC, *extra, "-c", src, "-o", obj]
    subprocess.run(cmd, check=True)
    return obj


# The phase-stamp variant: kernels record clock64 stamps per chunk of CTA 0 into the end of
# the workspace (KDA_PHASE_STAMPS); a separate library, never the one the package loads.
STAMPS_LIB = os.path.join(PKG, "libkda_stamps.so")


BINDING_SRC = os.path.join(CSRC, "kda_layer_binding.cpp")


def binding_path() -> str:
    """The marshalling module of ``layer.py``, one per torch version (its C++ ABI)."""
    import torch
    return os.path.join(PKG, "_layer_" + re.sub(r"\W+", "_", torch.__version__) + ".so")


def build_binding(force: bool = False) -> str:
    """Build (if stale) and return the path of the marshalling module."""
    import torch
    path = binding_path()
    deps = [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(path) and os.path.getmtime(path) >= max(map(os.path.getmtime, deps)):
        return path
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = (INCLUDE, sysconfig.get_paths()["include"], os.path.join(base, "include"),
            os.path.join(cuda, "include"))
    libs = os.path.join(base, "lib")
    tmp = path + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    *(x for d in dirs for x in ("-isystem", d)), BINDING_SRC, "-o", tmp, "-L", libs, "-lc10",
                    "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"], check=True)
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose_ptxas: bool = False, stamps: bool = False) -> str:
    """Build (if stale) and return the path of libkda.so (or of the stamps variant); with
    libkda.so, the marshalling module too."""
    path = _build_library(force, verbose_ptxas, stamps)
    if not stamps:
        build_binding(force)
    return path


def _build_library(force: bool, verbose_ptxas: bool, stamps: bool) -> str:
    lib = STAMPS_LIB if stamps else LIB
    bdir = BUILD + ("_stamps" if stamps else "")
    os.makedirs(bdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(lib):
        if os.path.getmtime(lib) >= max(os.path.getmtime(d) for d in deps):
            return lib
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    if stamps:
        extra = extra + ["-DKDA_PHASE_STAMPS"]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, bdir), srcs))
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
