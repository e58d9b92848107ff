"""Build libpoet.so in-tree for sm_100a with nvcc (no JIT; libpoet.so does not need torch).

    python -m orthogonal_reparameterized_poet_b200.build [--force]

Each .cu under csrc/ is compiled to an object under _build/ (in parallel),
then linked into orthogonal_reparameterized_poet_b200/libpoet.so.  Objects
are rebuilt when their source, a header, or this file is newer.  csrc/binding.cpp
becomes _binding.<python>.torch-<version>.so beside it (the host compiler, torch's
headers), the compiled binding of this interpreter and this torch.  Where it cannot
be compiled the build warns and goes on: every call works through ctypes too.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpoet.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, force):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if force or _stale(obj, [src] + _headers()):
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def binding_path() -> str:
    """Where the compiled binding for this interpreter and this torch lies: it uses their C++ interfaces, so one
    that was built for others must not be loaded."""
    import torch

    return os.path.join(PKG, f"_binding.{sys.implementation.cache_tag}.torch-{torch.__version__}.so")


def _binding(force):
    """The binding of the operators on torch tensors, linked against libpoet.so beside it."""
    src, path = os.path.join(CSRC, "binding.cpp"), binding_path()
    if not (force or _stale(path, [src] + _headers())):
        return
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(NVCC))
    include = cpp_extension.include_paths() + [os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in include], src,
           "-o", path, f"-L{PKG}", "-l:libpoet.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{r.stdout}\n{r.stderr}")


def _binding_if_possible(force):
    try:
        _binding(force)
    except (OSError, ImportError, RuntimeError) as e:
        warnings.warn(f"the compiled binding could not be built; calls go through ctypes:\n{e}")


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, force), srcs))
    if force or _stale(LIB, objs):
        cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", LIB, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _binding_if_possible(force)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
