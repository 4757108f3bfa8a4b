"""Build of the in-tree CUDA library (sm_100a) with nvcc.

``build()`` compiles ``csrc/la_lib.cu`` into ``_build/liblightning_attn.so``
next to this file; the Python binding loads it from there.  The library links
the CUDA runtime statically and reaches the driver (for TMA tensor maps) at run
time, so it loads on machines without a GPU.

It also compiles ``csrc/la_marshal.cpp`` with g++ against the headers of the
installed torch: a Python module that marshals the softmax calls' tensors in a
few microseconds less than Python code does.  Where it is missing (no compiler
or headers, another torch) the calls are marshalled in Python.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC_DIR = os.path.join(HERE, "csrc")
INCLUDE_DIR = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "liblightning_attn.so")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(SRC_DIR, "*.cu")) + glob.glob(os.path.join(SRC_DIR, "*.cuh"))
                  + [os.path.join(INCLUDE_DIR, "lightning_attn.h")])


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > t for s in sources())


def marshal_path() -> str:
    """The marshalling module built for this Python and torch."""
    import torch
    return os.path.join(BUILD_DIR, f"_marshal.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def build_marshal(force: bool = False) -> str | None:
    """Compile the marshalling module; None (with a warning) when that fails."""
    import torch
    src, path = os.path.join(SRC_DIR, "la_marshal.cpp"), marshal_path()
    deps = [src, os.path.join(INCLUDE_DIR, "lightning_attn.h")]
    if not force and os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps):
        return path
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE_DIR,
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           "-I", os.path.join(root, "include"), src, "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", BUILD_DIR, f"-l:{os.path.basename(LIB_PATH)}",
           "-Wl,-rpath,$ORIGIN"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        warnings.warn(f"the marshalling module was not built: {e}")
        return None
    if res.returncode != 0:
        warnings.warn("the marshalling module was not built:\n" + res.stderr[-2000:])
        return None
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not needs_build():
        build_marshal()
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-I", INCLUDE_DIR, "-I", SRC_DIR, *extra_flags,
           os.path.join(SRC_DIR, "la_lib.cu"), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)
    build_marshal(force)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
