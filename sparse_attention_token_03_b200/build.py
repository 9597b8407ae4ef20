"""Build libdsa_index.so in-tree with nvcc for sm_100a (no torch JIT cache), and
_serve_binding-*.so, the native host side of the serving calls, with g++."""

from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
INCLUDE = PKG.parent / "include"
LIB = PKG / "libdsa_index.so"
BINDING_SRC = PKG / "serve_binding.cpp"


def binding_path(torch_version: str, python_tag: str) -> Path:
    """The object inlines torch's C++ layouts and CPython's API: one per version of both."""
    return PKG / f"_serve_binding-{python_tag}-torch{torch_version}.so"


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # the library itself builds without it
        return "-none"


BINDING = binding_path(_torch_version(), sys.implementation.cache_tag)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared",
    "--expt-relaxed-constexpr",
]


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _inputs() -> list[Path]:
    return sources() + sorted(CSRC.glob("*.cuh")) + sorted(INCLUDE.glob("*.h"))


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found")


def stale() -> bool:
    if not LIB.exists():
        return True
    t = LIB.stat().st_mtime
    return any(p.stat().st_mtime > t for p in _inputs())


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile every .cu under csrc/ into one shared library next to this file."""
    if not force and not stale():
        return LIB
    tmp = LIB.with_suffix(f".{os.getpid()}.tmp")
    cmd = [nvcc(), *NVCC_FLAGS, f"-I{INCLUDE}", "-o", str(tmp), *map(str, sources())]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def binding_stale() -> bool:
    if not BINDING.exists():
        return True
    t = BINDING.stat().st_mtime
    return any(p.stat().st_mtime > t for p in (BINDING_SRC, *INCLUDE.glob("*.h")))


def build_binding(force: bool = False) -> Path:
    """Compile serve_binding.cpp against the installed torch and Python."""
    if not force and not binding_stale():
        return BINDING
    import sysconfig

    import torch

    tdir = Path(torch.__file__).parent
    cuda = Path(nvcc()).resolve().parent.parent
    tmp = BINDING.with_suffix(f".{os.getpid()}.tmp")
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        f"-I{tdir}/include", f"-I{tdir}/include/torch/csrc/api/include", f"-I{sysconfig.get_path('include')}",
        f"-I{cuda}/include", "-o", str(tmp), str(BINDING_SRC), f"-L{tdir}/lib",
        "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10_cuda", "-lc10",
    ])
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_binding(force="--force" in sys.argv))
