"""Build librmm.so in-tree with nvcc for sm_100a (B200).

    python -m input_adaptive_reduced_02_b200.build [--force]

Objects go to _build/ at the repository root; the shared library lands next to
this file so that the Python binding finds it. The CUDA runtime is linked
statically and the driver's tensor-map encoder is looked up at run time, so
the library loads on a host without a GPU.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "librmm.so")
SOURCES = ["api.cu", "score.cu", "select.cu", "pack.cu", "gemm_tc.cu", "gemm_simt.cu", "gemv.cu", "softmax.cu",
           "noalloc.cu", "attn.cu", "kv4.cu", "evict.cu", "api_attn.cu"]
HEADERS = ["rmm_device.cuh", "rmm_internal.h", "int8_convert.cuh", "api_common.h"]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O3", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _mtime(p):
    return os.path.getmtime(p) if os.path.exists(p) else -1.0


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    dep_time = max(_mtime(os.path.join(CSRC, h)) for h in HEADERS)
    dep_time = max(dep_time, _mtime(os.path.join(ROOT, "include", "rmm.h")), _mtime(__file__))
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _mtime(o) < max(_mtime(s), dep_time):
            cmd = [NVCC, *ARCH, *FLAGS, "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            subprocess.run(cmd, check=True)
    if force or _mtime(LIB) < max(_mtime(o) for o in objs):
        tmp = LIB + ".tmp"
        subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
        os.replace(tmp, LIB)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/shared-memory usage")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
