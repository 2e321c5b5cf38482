"""Build libmq.so (the CUDA kernels and the C ABI) in-tree with nvcc for sm_100a,
libmq_debug.so, the same sources with the bounds checks of MQ_DEBUG, and
_mq_torch.so, the native part of the binding (host code, against torch's headers).

Usage: python -m nvfp4_w4a4_quantized_03_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmq.so")
DEBUG_LIB = os.path.join(HERE, "libmq_debug.so")
TORCH_SRC = os.path.join(CSRC, "mq_torch.cpp")
TORCH_LIB = os.path.join(HERE, "_mq_torch.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(HERE, "..", "include", "mq.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _build_one(lib: str, objdir: str, extra, ptxas_verbose: bool) -> None:
    os.makedirs(objdir, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                    "-I", os.path.join(HERE, "..", "include")] + list(extra)
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        subprocess.check_call([nvcc(), "-c", src, "-o", obj] + flags)
        objs.append(obj)
    tmp = lib + ".tmp"
    subprocess.check_call([nvcc(), "-shared", "-o", tmp] + objs + ARCH + ["-lcudart_static"])
    os.replace(tmp, lib)


def _build_torch() -> None:
    """_mq_torch.so: calls libmq.so by address, so it links against torch alone."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = TORCH_LIB + ".tmp"
    subprocess.check_call(
        ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", TORCH_SRC, "-o", tmp,
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I", sysconfig.get_path("include"), "-I", os.path.join(cuda, "include"), "-I", os.path.join(root, "include"),
         "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
         "-Wl,-rpath," + os.path.join(root, "lib")])
    os.replace(tmp, TORCH_LIB)


def _torch_stale() -> bool:
    return not os.path.exists(TORCH_LIB) or any(
        os.path.getmtime(d) > os.path.getmtime(TORCH_LIB) for d in (TORCH_SRC, os.path.join(HERE, "..", "include", "mq.h")))


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Build the libraries whose sources are newer (or `force`); returns libmq.so's path."""
    if force or _stale(LIB):
        _build_one(LIB, os.path.join(HERE, "_build"), [], ptxas_verbose)
    if force or _stale(DEBUG_LIB):
        _build_one(DEBUG_LIB, os.path.join(HERE, "_build", "debug"), ["-DMQ_DEBUG=1"], ptxas_verbose)
    if force or _torch_stale():
        _build_torch()
    return LIB


if __name__ == "__main__":
    build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
