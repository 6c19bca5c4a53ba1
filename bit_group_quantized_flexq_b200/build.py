"""Builds the CUDA library libflexq.so in this package directory (sm_100a).

Usage: python -m bit_group_quantized_flexq_b200.build [--verbose]
"""

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "flexq_lib.cu")
LIB = os.path.join(PKG, "libflexq.so")
DEPS = [os.path.join(PKG, "csrc", f) for f in
        ("flexq_lib.cu", "flexq_api.cu", "flexq_gemm.cuh", "flexq_gemm_wide.cuh",
         "flexq_quant.cuh", "flexq_ptx.cuh", "flexq_w4.cuh", "flexq_w4_gemm.cuh",
         "flexq_embed.cuh", "flexq_w4_api.cuh")] + \
       [os.path.join(ROOT, "include", "flexq.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
]


def nvcc_path():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def build(force=False, verbose=False):
    """Compile libflexq.so unless it is newer than every source; returns its path."""
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc_path()] + NVCC_FLAGS + ["-o", tmp, SRC]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    if verbose:
        sys.stdout.write(r.stdout + r.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="--verbose" in sys.argv))
