"""Build libbitdelta.so in-tree for sm_100a with nvcc (no JIT, no torch extension).

    python -m tenant_serving_b200.build          # or: python tenant_serving_b200/build.py
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libbitdelta.so")
SOURCES = ["bd_abi.cu", "bd_compress.cu", "bd_reconstruct.cu", "bd_apply.cu", "bd_base_tc.cu",
           "bd_prepare.cu", "bd_delta_tc.cu", "bd_delta_lut.cu", "bd_cache.cu",
           "bd_base_fp8.cu", "bd_fp4.cu", "bd_mm_fp4.cu", "bd_gemv_fp4.cu", "bd_delta_fp4.cu"]
HEADERS = ["bd_internal.cuh", "bd_tc.cuh", "bd_fp4.cuh", "bd_fp4_mma.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(OUT):
        return True
    t = os.path.getmtime(OUT)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "bitdelta.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not _stale():
        return OUT
    cmd = [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--shared",
           "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), "-o", OUT + ".tmp"]
    if ptxas_info:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(CSRC, f) for f in SOURCES]
    if verbose:
        print(" ".join(cmd))
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + r.stdout + r.stderr)
    if verbose or ptxas_info:
        sys.stdout.write(r.stdout + r.stderr)
    os.replace(OUT + ".tmp", OUT)
    return OUT


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(OUT)
