"""Builds libqsa_b200.so (the CUDA kernels and the C ABI) in-tree with nvcc,
and _qsa_torch.<tag>.so (the short way from PyTorch tensors to it) with g++.

    python -m token_indexed_sparse_b200.build [--force]

The library is compiled for sm_100a only and links the CUDA runtime statically,
so it carries no dependency on the runtime bundled with PyTorch, and it is built
without one too.  The binding is compiled against the PyTorch that imports it; the
tag in its name is that PyTorch's, so one built for another is never loaded.
Without a binding the same calls go their longer way through Python.
"""

from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqsa_b200.so")
BINDING_SOURCE = os.path.join(CSRC, "qsa_torch.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["qsa_api.cu", "qsa_routes.cu", "qsa_forward.cu", "qsa_backward.cu", "qsa_noalloc.cu", "qsa_bitmap.cu", "qsa_selector.cu", "qsa_dkdv_union.cu", "qsa_cast.cu",
           "qsa_rope.cu", "qsa_paged.cu", "qsa_causal.cu", "qsa_cache_api.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the QSA library needs the CUDA 12.9 toolkit to build")


def _inputs():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "qsa.h")]
    return [d for d in deps if d != BINDING_SOURCE]


def _newer(out: str, inputs) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def binding_path() -> str:
    """The binding's file for the installed PyTorch and Python."""
    import torch

    made_for = "|".join(str(x) for x in (torch.__version__, torch.version.git_version,
                                         torch._C._GLIBCXX_USE_CXX11_ABI, sysconfig.get_config_var("SOABI")))
    return os.path.join(PKG, f"_qsa_torch.{hashlib.sha256(made_for.encode()).hexdigest()[:12]}.so")


def build_binding(force: bool = False) -> str:
    """Compiles the binding against the installed PyTorch; raises where that fails."""
    binding = binding_path()
    if not force and _newer(binding, [BINDING_SOURCE, os.path.join(INCLUDE, "qsa.h")]):
        return binding
    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    includes = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"),
                *cpp_extension.include_paths()]
    tmp = binding + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in includes], BINDING_SOURCE, "-o", tmp,
           *[f"-L{p}" for p in cpp_extension.library_paths()], "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, binding)
    return binding


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, and the binding where there is a PyTorch that it compiles against (else a warning says so)."""
    lib = build_library(force, verbose)
    try:
        build_binding(force)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn(f"the library is built, the PyTorch binding is not (the paged-cache calls of qsa.py go their "
                      f"longer way): {e}", RuntimeWarning, stacklevel=2)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = []
    log = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log.append(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(os.path.join(BUILD_DIR, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    if verbose:
        print("\n".join(log))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
