"""Build the sm_100a shared library ``libivit_b200.so`` in-tree with nvcc, and
the native part of the Python binding, ``_binding.<torch>.<Python ABI>.so``,
with g++.

    python -m integer_only_quantized_int8_b200.build [--verbose]
    python integer_only_quantized_int8_b200/build.py --library [--verbose]

The second form builds the C library alone and needs nothing but nvcc; the
binding also takes torch's and Python's headers.  The library links the CUDA runtime statically and resolves the one driver
entry point it needs (tensor-map encoding) at run time, so it loads on a
machine without a GPU driver; compute calls then return IVIT_ERR_CUDA.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libivit_b200.so")
BINDING_SRC = os.path.join(PKG, "csrc", "binding.cpp")
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "-shared", "-cudart", "static",
    "--expt-relaxed-constexpr", "--threads", "8",
]


def sources():
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(PKG, "csrc", "*.cuh"))) + \
        sorted(glob.glob(os.path.join(PKG, "csrc", "*.h"))) + sorted(glob.glob(os.path.join(ROOT, "include", "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in deps())


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def binding_path() -> str:
    """The binding of the running Python and torch.  It uses torch's C++ classes, whose layout changes between
    versions, so a file of another version is never the one loaded."""
    import torch
    version = "".join(ch if ch.isalnum() or ch == "." else "_" for ch in torch.__version__)
    return os.path.join(PKG, f"_binding.torch-{version}" + sysconfig.get_config_var("EXT_SUFFIX"))


def binding_deps():
    return [BINDING_SRC, os.path.join(ROOT, "include", "ivit.h")]


def build_binding(force: bool = False) -> str:
    path = binding_path()
    if not force and os.path.exists(path) and os.path.getmtime(path) >= max(map(os.path.getmtime, binding_deps())):
        return path
    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [base, os.path.join(base, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
                os.path.join(cuda, "include")]
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in includes), "-o", tmp, BINDING_SRC,
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"g++ failed building {os.path.basename(path)} (the C library needs no g++ and is built)")
    os.replace(tmp, path)
    return path


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include")]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += ["-o", tmp, *sources()]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libivit_b200.so")
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


def build(force: bool = False, verbose: bool = False) -> str:
    build_library(force, verbose)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    (build_library if "--library" in sys.argv else build)(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
