"""Build the sm_100a shared library ``libschnet_b200.so`` in-tree with nvcc, and
the Python binding of its readout-tuning calls, ``_binding.so``, with g++.

Usage: ``python -m schnet_gnn_molecular_b200.build [--force] [--verbose] [--library-only]``.
The library exports the C ABI declared in ``include/schnet.h``; building it alone (``--library-only``, or without
PyTorch installed) needs nvcc only.
"""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libschnet_b200.so")
SOURCES = ["api.cu", "neighbors.cu", "cfconv.cu", "atomwise.cu", "integrate.cu", "taps.cu", "readout.cu",
           "preference.cu"]
HEADERS = ["common.cuh", "internal.h", os.path.join("..", "..", "include", "schnet.h")]

CUDA_DEFAULT = "/usr/local/cuda"
NVCC = os.environ.get("NVCC", os.path.join(CUDA_DEFAULT, "bin", "nvcc"))
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "-ftz=true",
         "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr", "-Xcompiler", "-fvisibility=hidden"]


BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCES = ["binding.cpp", os.path.join("..", "..", "include", "schnet.h")]


def _stale(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, s) for s in sources] + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def built_for() -> str:
    """What a binding fits beside its sources: this PyTorch and this interpreter."""
    return f"torch {importlib.metadata.version('torch')} {sys.implementation.cache_tag}"


def _other_torch() -> bool:
    """Whether the binding was built for another PyTorch or interpreter (its note, beside it, says which)."""
    try:
        with open(BINDING + ".txt") as f:
            return f.read() != built_for()
    except OSError:
        return True


def cuda_include() -> str:
    """The folder of CUDA's headers: nvcc's own, whether NVCC is a path, a link or a name on PATH; else CUDA_HOME's."""
    nvcc = shutil.which(NVCC)
    homes = [os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))] if nvcc else []
    for home in [*homes, os.environ.get("CUDA_HOME"), CUDA_DEFAULT]:
        if home and os.path.exists(os.path.join(home, "include", "cuda_runtime_api.h")):
            return os.path.join(home, "include")
    raise RuntimeError(f"no cuda_runtime_api.h beside {NVCC}, in CUDA_HOME or in {CUDA_DEFAULT}")


def _build_binding(verbose: bool) -> None:
    import sysconfig

    import torch
    top = os.path.dirname(torch.__file__)
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for d in (os.path.join(top, "include"), os.path.join(top, "include", "torch", "csrc", "api", "include"),
                         cuda_include(), sysconfig.get_paths()["include"]) for x in ("-isystem", d)],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", HERE, "-l:" + os.path.basename(LIB),
           "-L", os.path.join(top, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)


def _have_torch() -> bool:
    try:
        return bool(built_for())
    except importlib.metadata.PackageNotFoundError:
        return False


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None, binding: bool = True) -> str:
    """binding = False, or no PyTorch: the library alone, which is all that a user of the C ABI needs."""
    if force or _stale(LIB, SOURCES + HEADERS):
        _build_library(verbose, extra)
    if not binding or not _have_torch():
        return LIB
    if force or _stale(BINDING, BINDING_SOURCES) or _other_torch():
        _build_binding(verbose)
        with open(BINDING + ".txt", "w") as f:
            f.write(built_for())
    return LIB


def _build_library(verbose: bool, extra: list[str] | None) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *FLAGS, *(extra or []), "-I", os.path.join(ROOT, "include"),
           *[os.path.join(CSRC, s) for s in SOURCES], "-o", tmp, "-lcuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else None
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv or extra is not None, extra=extra,
                binding="--library-only" not in sys.argv))
