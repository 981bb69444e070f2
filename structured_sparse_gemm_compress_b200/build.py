"""Build libnmspmm.so (sm_100a) in-tree with nvcc, and the compiled Python binding
of the feed-forward calls (_binding.so) with g++ against torch's headers.

Usage: python -m structured_sparse_gemm_compress_b200.build [--force] [-v] [--trace]

--trace also builds libnmspmm_trace.so: the same sources compiled with
NM_TRACE, whose SpMM kernels record per-CTA pipeline timestamps into a buffer
named by NMSPMM_TRACE_PTR (see trace.py).  The product library never has them.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(PKG, "libnmspmm.so")
TRACE_LIB = os.path.join(PKG, "libnmspmm_trace.so")
BINDING = os.path.join(PKG, "_binding.so")
OBJDIR = os.path.join(PKG, "_build")
TRACE_OBJDIR = os.path.join(PKG, "_build_trace")
SOURCES = ["nm_api.cu", "nm_pack.cu", "nm_spmm.cu", "nm_gated.cu", "nm_grad.cu", "nm_mx.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-std=c++17", "-lineinfo",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    deps = [src] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    deps.append(os.path.join(INCLUDE, "nmspmm.h"))
    return any(os.path.getmtime(d) > os.path.getmtime(obj) for d in deps)


def _compile(src: str, force: bool, extra: list[str], objdir: str = OBJDIR) -> str:
    obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
    path = os.path.join(CSRC, src)
    if force or _stale(obj, path):
        subprocess.check_call([NVCC, *FLAGS, *extra, "-c", path, "-o", obj])
    return obj


def _binding(force: bool) -> str:
    """_binding.so: csrc/nm_binding.cpp against torch's C++ library (rebuilt for another torch or Python)."""
    import sysconfig

    import torch

    src, stamp = os.path.join(CSRC, "nm_binding.cpp"), os.path.join(OBJDIR, "binding.torch")
    built_for = open(stamp).read() if os.path.exists(stamp) else ""
    wanted = f"{torch.__version__} {sysconfig.get_config_var('SOABI')}"
    if force or _stale(BINDING, src) or built_for != wanted:
        root = os.path.dirname(torch.__file__)
        dirs = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), sysconfig.get_paths()["include"]]
        tmp = BINDING + f".{os.getpid()}.tmp"
        subprocess.check_call([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
                               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                               *(a for d in dirs for a in ("-isystem", d)), src, "-o", tmp,
                               "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
                               "-ltorch_cuda", "-lc10", "-lc10_cuda"])
        os.replace(tmp, BINDING)
        with open(stamp, "w") as f:
            f.write(wanted)
    return BINDING


def build(force: bool = False, verbose_ptxas: bool = False, trace: bool = False) -> str:
    lib, objdir = (TRACE_LIB, TRACE_OBJDIR) if trace else (LIB, OBJDIR)
    os.makedirs(objdir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    if trace:
        extra.append("-DNM_TRACE")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if trace else ex.submit(_binding, force)
        objs = list(ex.map(lambda s: _compile(s, force, extra, objdir), SOURCES))
    if force or not os.path.exists(lib) or any(os.path.getmtime(o) > os.path.getmtime(lib) for o in objs):
        tmp = lib + f".{os.getpid()}.tmp"
        subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs,
                               "-o", tmp, "-lcudart"])
        os.replace(tmp, lib)
    if binding is not None and binding.exception() is not None:  # the C library needs none of it: it is there
        raise RuntimeError(f"{lib} is built, but not the Python binding, which needs {CXX} and torch's "
                           f"headers: {binding.exception()}") from binding.exception()
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
    if "--trace" in sys.argv:
        print(build(force="--force" in sys.argv, trace=True))
