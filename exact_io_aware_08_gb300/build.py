"""Build libfa.so in-tree from csrc/*.cu for sm_103a, and the extension module from csrc/binding.cpp.

Each translation unit is compiled in parallel with nvcc, then linked into
``exact_io_aware_08_gb300/libfa.so`` (git-ignored); the extension module is compiled beside them with
g++ against the installed torch's headers.  Rebuilds only when a source or header is newer than what
it makes.  Usage: ``python -m exact_io_aware_08_gb300.build [--force] [-v] [--no-binding]``.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                 "-I" + os.path.join(ROOT, "include"), "-diag-suppress", "177"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + [os.path.join(ROOT, "include", "fa.h"), os.path.abspath(__file__)])


def _newer(made, deps) -> bool:
    return os.path.exists(made) and all(os.path.getmtime(p) <= os.path.getmtime(made) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def binding_path() -> str:
    """Where the extension module lies.  It is made of torch's C++ classes and Python's: its name says of
    which, so that another torch or Python finds none and has it built."""
    import torch
    made_of = f"{sys.implementation.cache_tag}-torch{torch.__version__}-abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return os.path.join(HERE, f"_binding-{made_of}.so")


def binding_up_to_date() -> bool:
    return _newer(binding_path(), [BINDING_SOURCE, os.path.join(ROOT, "include", "fa.h"), os.path.abspath(__file__)])


def build_binding() -> str:
    """Compile the extension module."""
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(home, "lib")
    path = binding_path()
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-o", tmp, BINDING_SOURCE,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-I" + i for i in include), "-L" + lib,
           "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=(), binding: bool = True) -> str:
    """Build what is out of date.  ``binding=False``: libfa.so alone, which needs no torch.  A module that
    does not compile is an error, but libfa.so is made all the same."""
    lib_stale = force or not up_to_date()
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(lambda: None if not force and binding_up_to_date() else build_binding()) if binding else None
        if lib_stale:
            _build_library(verbose, extra_flags)
    if module is not None:
        module.result()
    return LIB


def _build_library(verbose, extra_flags):
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [nvcc, *CFLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, binding="--no-binding" not in sys.argv)
    print(LIB)
