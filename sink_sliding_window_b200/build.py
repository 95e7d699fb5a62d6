"""Builds libsinkattn.so (the C-ABI library) in-tree with nvcc for sm_100a, and
the native binding of its paged-cache calls (binding_path()) if torch is there.

    python -m sink_sliding_window_b200.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsinkattn.so")
BINDING_SRC = os.path.join(CSRC, "paged_binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(target, sources) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in sources)


def up_to_date() -> bool:
    return _newer(LIB, _sources())


def binding_path() -> str:
    """The native binding's file, which names the interpreter and the torch that
    it is compiled for: neither promises the next version its binary interface."""
    import torch
    return os.path.join(PKG, f"_paged.{sys.implementation.cache_tag}.torch-{torch.__version__}.so")


def build_binding(force: bool = False) -> str:
    """The binding, compiled by the host compiler against torch's headers; it
    finds libsinkattn.so beside it."""
    import torch
    target, header = binding_path(), os.path.join(INCLUDE, "sink_attn.h")
    if not force and _newer(target, [BINDING_SRC, header]):
        return target
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    tmp = target + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(cuda, "include"),
           "-isystem", sysconfig.get_paths()["include"], BINDING_SRC, "-o", tmp, "-L", PKG, "-l:" + os.path.basename(LIB),
           "-L", os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, target)
    return target


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    if force or not up_to_date():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
               "-Xcompiler", "-fPIC", "-shared", "-I", INCLUDE, "-I", CSRC,
               os.path.join(CSRC, "sink_attn.cu"), "-o", tmp]
        if ptxas_verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    try:
        import torch  # noqa: F401
    except ImportError:
        return LIB  # complete for programs in C; the binding is torch's
    build_binding(force)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas))


if __name__ == "__main__":
    sys.exit(main())
