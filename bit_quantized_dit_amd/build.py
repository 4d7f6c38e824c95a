"""Build the gfx950 HIP library (libw4a4.so) in-tree with hipcc.

Run ``python -m bit_quantized_dit_amd.build`` (or ``__graft_entry__.build()``).  The
shared library lands next to this file, where the ctypes binding looks for it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libw4a4.so")
SOURCES = ["capi.hip", "calib.hip", "pack.hip", "actprep.hip", "gemm.hip", "gelu.hip", "search.hip", "dynamic.hip",
           "fp8_capi.hip", "fp8.hip", "fp8gemm.hip", "moe.hip", "int8_capi.hip", "int8.hip", "int8gemm.hip",
           "kv_capi.hip", "kv.hip", "kvattn.hip"]

# Numerics-relevant flags: IEEE binary32 division, fp32 subnormals kept, no FMA
# contraction, no fast-math; packed-fp32 instructions disabled.
HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm not installed?)")


def build_library(verbose: bool = False) -> str:
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", os.path.join(HERE, "..", "include"), "-o", tmp, *srcs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library(verbose="-v" in sys.argv))
