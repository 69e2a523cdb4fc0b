"""Build libdiffattn.so (sm_100a) in-tree with nvcc, and the binding's
marshalling module (_marshal.so) with the host compiler.

Usage: python -m differential_attention_sm_b200.build [--force]
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdiffattn.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
MARSHAL = os.path.join(PKG, "_marshal.so")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-Xptxas", "-v",
    "-I" + INCLUDE,
]
# The CUDA-core kernels in simt.cu serve the fp32 workload, whose accuracy
# bound (1e-5 max abs) leaves no room for approximate exp, division and
# square root: that file is built with IEEE-compliant math, and so is
# qk_norm_rope.cu, whose fp32 rows are held to fp32's own steps.  Every other file
# uses fast math (its exponentials are explicit ex2.approx or polynomial).
PRECISE = {"simt.cu", "qk_norm_rope.cu"}


def flags_for(src: str):
    return FLAGS + ([] if os.path.basename(src) in PRECISE else ["--use_fast_math"])


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [
        os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ into one shared library, and the binding's
    marshalling module; returns the library's path."""
    build_marshal(force)
    if not force and not _stale():
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *flags_for(src), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s" % os.path.basename(src))
        objs.append(obj)
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
           "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("link of libdiffattn.so failed")
    os.replace(tmp, LIB)
    return LIB


def build_marshal(force: bool = False) -> str:
    """Compile the binding's marshalling module against the installed torch;
    returns its path."""
    import torch
    src = os.path.join(CSRC, "marshal.cpp")
    stamp = os.path.join(PKG, "_build", "marshal.torch")   # its C++ interface is torch's
    built = open(stamp).read() if os.path.exists(stamp) else ""
    deps = (src, os.path.join(INCLUDE, "diffattn.h"))
    if (not force and built == torch.__version__ and os.path.exists(MARSHAL) and
            all(os.path.getmtime(d) <= os.path.getmtime(MARSHAL) for d in deps)):
        return MARSHAL
    os.makedirs(os.path.dirname(stamp), exist_ok=True)
    root = os.path.dirname(torch.__file__)
    tmp = MARSHAL + ".%d.tmp" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared",
           "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           '-DDA_TORCH_VERSION="%s"' % torch.__version__,
           "-I" + sysconfig.get_paths()["include"], "-I" + INCLUDE,
           "-I" + os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           src, "-o", tmp, "-L" + os.path.join(root, "lib"),
           "-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("the host compiler failed on marshal.cpp")
    os.replace(tmp, MARSHAL)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return MARSHAL


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
