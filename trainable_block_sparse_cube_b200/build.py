"""Builds libvsa.so in-tree with nvcc for sm_100a.

Usage: python -m trainable_block_sparse_cube_b200.build
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
SRC = ["api.cu", "gather.cu", "coarse.cu", "fine.cu", "measure.cu", "backward.cu", "fine_bwd.cu", "schedule.cu",
       "rope.cu", "api_project.cu", "linear.cu", "api_linear.cu"]
LIB = os.path.join(HERE, "libvsa.so")
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "static",
]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    raise RuntimeError("nvcc not found")


def build(verbose: bool = False, force: bool = False) -> str:
    srcs = [os.path.join(HERE, "csrc", s) for s in SRC]
    deps = srcs + [os.path.join(HERE, "csrc", h) for h in ("vsa_common.cuh", "sm100_ptx.cuh", "pair_ptx.cuh", "host.cuh",
                                                            "packed.cuh", "launch.cuh")]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "vsa.h"))
    if not force and os.path.exists(LIB):
        t = os.path.getmtime(LIB)
        if all(os.path.getmtime(d) <= t for d in deps):
            return LIB
    cmd = [_nvcc(), *NVCC_FLAGS, "-o", LIB + ".tmp", *srcs]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
