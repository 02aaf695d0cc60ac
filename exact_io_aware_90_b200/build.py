"""Builds libfa_b200.so in-tree with nvcc for sm_100a, and the torch binding of the wrappers (_binding.so) with g++.

Usage: python exact_io_aware_90_b200/build.py [--verbose-ptxas]   (by path: importing the package would load the
existing library first)
Both land next to this file; the Python package loads them from there.
"""
from __future__ import annotations

import json
import os
import shutil
import subprocess
import sys
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB_NAME = "libfa_b200.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BINDING_PATH = os.path.join(HERE, "_binding.so")
BUILT_FOR_PATH = os.path.join(HERE, "_binding.json")  # the interpreter and torch that _binding.so was built for
SOURCES = ["libfa_b200.cu"]
DEPS = ["fa_api.cu", "fa_fwd.cu", "fa_bwd.cu", "fa_decode.cu", "fa_merge.cu", "fa_noalloc.cu", "fa_rope.cu",
        "fa_cache.cu", "fa_paged.cu", "fa_paged_api.cu"]
HEADERS = ["fa_internal.h", "sm100.cuh", "fa_paged_internal.h", "async_copy.cuh", "rope.cuh", "paged.cuh", os.path.join("..", "..", "include", "fa.h")]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: set NVCC or put the CUDA toolkit on PATH")


def _older(path: str, deps) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def needs_rebuild() -> bool:
    return _older(LIB_PATH, [os.path.join(CSRC, f) for f in SOURCES + DEPS + HEADERS] + [__file__])


def _built_for() -> dict:
    import torch
    return {"python": sys.version, "torch": str(torch.__version__), "torch_git": str(torch.version.git_version),
            "cuda": str(torch.version.cuda), "cxx11_abi": int(torch._C._GLIBCXX_USE_CXX11_ABI)}


def binding_needs_rebuild() -> bool:
    """Older than its sources, or built for another interpreter or torch: their C++ ABI differs."""
    if _older(BINDING_PATH, [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "fa.h"), __file__]):
        return True
    try:
        with open(BUILT_FOR_PATH) as f:
            return json.load(f) != _built_for()
    except (OSError, ValueError):
        return True


def build_binding(force: bool = False) -> Optional[str]:
    """The torch binding: linked against this interpreter's torch and, by a path relative to itself, the library.  Without
    torch there is none: the library is for use through its C ABI then."""
    try:
        import torch
    except ImportError:
        sys.stderr.write("torch is not installed: " + os.path.basename(BINDING_PATH) + " (the wrappers of paged.py) is not built\n")
        return None
    import sysconfig
    src = os.path.join(CSRC, "binding.cpp")
    if not force and not binding_needs_rebuild():
        return BINDING_PATH
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    # the system compiler, not $CXX: a toolchain that links libstdc++ in statically breaks against torch's shared one
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda,
           "-I", sysconfig.get_paths()["include"], src, "-o", BINDING_PATH + ".tmp",
           "-L", libs, "-L", HERE, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lfa_b200",
           "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building " + os.path.basename(BINDING_PATH))
    os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
    with open(BUILT_FOR_PATH + ".tmp", "w") as f:
        json.dump(_built_for(), f)
    os.replace(BUILT_FOR_PATH + ".tmp", BUILT_FOR_PATH)
    return BINDING_PATH


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    if not force and not needs_rebuild():
        build_binding()
        return LIB_PATH
    cmd = [
        nvcc_path(),
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-O3", "-lineinfo", "-std=c++17",
        "-Xcompiler", "-fPIC", "-shared",
        "--expt-relaxed-constexpr",
        "-I", os.path.join(ROOT, "include"),
        "-o", LIB_PATH + ".tmp",
    ] + [os.path.join(CSRC, f) for f in SOURCES]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building " + LIB_NAME)
    if verbose_ptxas:
        sys.stderr.write(res.stderr)
    os.replace(LIB_PATH + ".tmp", LIB_PATH)
    build_binding(force)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose_ptxas="--verbose-ptxas" in sys.argv, force=True))
