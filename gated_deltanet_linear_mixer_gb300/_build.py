"""Builds libgdn.so (the CUDA kernels + C ABI) in-tree with nvcc for sm_103a, and
_gdn_bind.so (the native argument marshalling of paged.py) with g++.

Each translation unit is compiled in parallel, then linked into one shared
library next to this file.  Rebuilds only when a source or header is newer than
the libraries, or the module was built for another PyTorch or Python.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libgdn.so")
BIND_SRC = os.path.join(CSRC, "gdn_bind.cpp")
BIND_PATH = os.path.join(PKG, "_gdn_bind.so")
BIND_STAMP = os.path.join(BUILD_DIR, "bind.txt")  # what _gdn_bind.so was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libgdn.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(INCLUDE, "gdn.h"), BIND_SRC, __file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BIND_PATH):
        return False
    if not os.path.exists(BIND_STAMP) or open(BIND_STAMP).read() != _bind_for():
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BIND_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _bind_for() -> str:
    """The PyTorch and the Python that the binding's module is tied to."""
    import torch
    return f"{torch.__version__} {os.path.dirname(torch.__file__)} {sysconfig.get_config_var('EXT_SUFFIX')}"


def _bind_flags():
    """Include and link flags of a CPython module on top of this PyTorch."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    compile_flags = ["-O2", "-std=c++17", "-fPIC", "-DUSE_CUDA",
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                     "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
                     "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
                     "-I", INCLUDE]
    link_flags = ["-shared", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                  "-L", PKG, "-lgdn", f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]
    return compile_flags, link_flags


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every csrc/*.cu for sm_103a and link libgdn.so; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    def run(what, cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    cxx = os.environ.get("CXX") or "g++"
    bind_compile, bind_link = _bind_flags()
    bind_obj = os.path.join(BUILD_DIR, "gdn_bind.cpp.o")
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        bind = ex.submit(run, "g++ on gdn_bind.cpp", [cxx, *bind_compile, "-c", BIND_SRC, "-o", bind_obj])
        objs = list(ex.map(compile_one, srcs))
        bind.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    run("link of libgdn.so", [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    os.replace(tmp, LIB_PATH)
    tmp = BIND_PATH + f".tmp{os.getpid()}"
    run("link of _gdn_bind.so", [cxx, bind_obj, "-o", tmp, *bind_link])
    os.replace(tmp, BIND_PATH)
    with open(BIND_STAMP, "w") as f:
        f.write(_bind_for())
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
