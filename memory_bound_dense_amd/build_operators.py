"""Build libmbd_operators.so, the operators around the GEMV, in-tree.

    python -m memory_bound_dense_amd.build_operators [-v]

A library of its own (include/operators.h), so the GEMV's stays what its
committed profiles were taken on.  Its many kernel forms are compiled side by
side, one object per source, and linked against libgemv.so (its handles and status
strings), which has to be there.  The flags are the GEMV library's.
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

from .build import ARCH, CSRC, INCLUDE, PKG, hipcc

LIB = os.path.join(PKG, "libmbd_operators.so")
# the longest first
SOURCES = [os.path.join(CSRC, f) for f in (
    "gla_scan_out_f16.hip", "gla_scan_out_bf16.hip", "gla_scan_grad_f16.hip", "gla_scan_grad_bf16.hip",
    "gla_scan_state_f16.hip", "gla_scan_state_bf16.hip", "gemm.hip", "gla_scan.hip", "rmsnorm.hip",
    "operators.hip")]
FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-mllvm", "-amdgpu-kernarg-preload-count=16", "-I", INCLUDE, "-I", CSRC]


def build(verbose: bool = False) -> str:
    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as d:
        objects = [os.path.join(d, os.path.basename(s) + ".o") for s in SOURCES]
        jobs = max(1, min(len(SOURCES), int(os.environ.get("MAX_JOBS", "8"))))
        with ThreadPoolExecutor(jobs) as pool:
            list(pool.map(lambda so: run([hipcc()] + FLAGS + ["-c", so[0], "-o", so[1]]),
                          zip(SOURCES, objects)))
        run([hipcc(), "--offload-arch=" + ARCH, "-fPIC", "-shared"] + objects +
            ["-L", PKG, "-lgemv", "-Wl,-rpath,$ORIGIN", "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
