"""Build libblin.so (C ABI + sm_100a kernels) with nvcc and its tensor-side extension with g++, in place.

    python block_causal_linear_rope_b200/build.py [--force] [--verbose-ptxas]

(Run as a script: importing the package itself loads the library.)
"""
from __future__ import annotations

import argparse
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libblin.so")
EXT = os.path.join(PKG, "_blin_torch.so")  # tensor-side marshalling (links libblin.so and torch)
EXT_SRC = os.path.join(CSRC, "blin_torch.cpp")
EXT_FOR = os.path.join(CSRC, "_build", "blin_torch.for")  # the torch and Python that it was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCES = ["blin_api.cu", "blin_kernels.cu", "blin_noalloc.cu", "blin_tconv.cu", "blin_decay.cu",
           "blin_rope.cu"]
FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + glob.glob(os.path.join(CSRC, "*.cuh")) +
            [os.path.join(ROOT, "include", "blin.h")])


def build_ext(force: bool = False) -> str:
    """The CPython extension that checks tensors and calls the library."""
    import sysconfig

    import torch
    srcs = [EXT_SRC, os.path.join(ROOT, "include", "blin.h")]
    now = f"torch {torch.__version__} at {os.path.dirname(torch.__file__)}, Python {sys.version}"
    if not force and os.path.exists(EXT) and all(os.path.getmtime(p) <= os.path.getmtime(EXT) for p in srcs):
        if os.path.exists(EXT_FOR) and open(EXT_FOR).read() == now:
            return EXT
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = EXT + f".tmp{os.getpid()}"
    lib = os.path.join(base, "lib")
    subprocess.check_call([
        os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wno-attributes",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{i}" for i in inc], EXT_SRC, "-o", tmp,
        f"-L{PKG}", "-l:libblin.so", f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
        "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"])
    os.replace(tmp, EXT)
    os.makedirs(os.path.dirname(EXT_FOR), exist_ok=True)
    with open(EXT_FOR, "w") as f:
        f.write(now)
    return EXT


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and not needs_build():
        build_ext()
        return LIB
    objs = []
    for src in SOURCES:
        obj = os.path.join(CSRC, "_build", src.replace(".cu", ".o"))
        os.makedirs(os.path.dirname(obj), exist_ok=True)
        cmd = [NVCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_verbose:
            cmd += ["-Xptxas", "-v"]
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    build_ext(force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.verbose_ptxas))
    sys.exit(0)
