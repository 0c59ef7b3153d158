"""Builds libgbs.so (all CUDA sources under csrc/) in-tree for sm_100a.

Usage: python -m gated_block_sparse_gate_b200.build [--force] [--debug]
The library is rebuilt when any source or header is newer than it. --debug
builds libgbs_debug.so instead: the same sources with -DGBS_DEBUG, whose
kernels check every index they read from a list and report a bad one as
GBS_ERR_DEVICE_CHECK (a stand-in for a device memory checker).
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgbs.so")
DEBUG_LIB = os.path.join(HERE, "libgbs_debug.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib=LIB):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(f) > t for f in deps)


def marshal_path() -> str:
    """Where the binding's native module for this Python and this torch is: its code is compiled against torch's
    own structures, so the name holds torch's version and commit. Raises ImportError without torch."""
    import torch

    tag = re.sub(r"[^\w.+]", "_", f"{torch.__version__}-{(torch.version.git_version or '')[:8]}")
    return os.path.join(HERE, f"_marshal-{tag}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_marshal(force: bool = False, verbose: bool = False):
    """The binding's argument checks and calls on the tensors themselves (csrc/marshal.cpp),
    where torch, its headers, Python's and CUDA's and a host compiler are installed. Where one
    is missing or the compiler fails, that is said and None returned: the binding does the same
    in Python."""
    src = os.path.join(CSRC, "marshal.cpp")
    try:
        import torch
        from torch.utils import cpp_extension

        module = marshal_path()
    except ImportError:
        return None
    if not force and os.path.exists(module) and os.path.getmtime(module) > max(
            map(os.path.getmtime, (src, os.path.join(INCLUDE, "gbs.h")))):
        return module
    include = sysconfig.get_paths()["include"]
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    dirs = [include, *cpp_extension.include_paths(), cuda, INCLUDE]
    if not all(any(os.path.exists(os.path.join(d, h)) for d in dirs)
               for h in ("Python.h", "torch/csrc/autograd/python_variable.h", "c10/cuda/CUDAStream.h",
                         "cuda_runtime_api.h")):
        return None
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(x for d in dirs for x in ("-isystem", d)), src, "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", module + ".tmp"]
    if verbose:
        print(" ".join(cmd))
    try:
        subprocess.run(cmd, check=True)
    except (OSError, subprocess.CalledProcessError) as e:
        if os.path.exists(module):  # of other sources
            os.remove(module)
        warnings.warn(f"csrc/marshal.cpp was not built ({e}); the binding checks arguments in Python")
        return None
    os.replace(module + ".tmp", module)
    return module


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    lib = build_library(force, verbose, debug)
    build_marshal(force, verbose)
    return lib


def build_library(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """The C library, which needs nvcc only."""
    lib = DEBUG_LIB if debug else LIB
    if not force and not _stale(lib):
        return lib
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = lib + ".tmp"
    flags = NVCC_FLAGS + (["-DGBS_DEBUG"] if debug else [])
    cmd = [nvcc, *flags, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *sources()]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv))
