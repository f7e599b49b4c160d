"""Builds the HIP library libob.so in-tree for gfx950 with hipcc.

Run as ``python -m error_compensated_bit_02_amd.build``.  The flags matter for
correctness: fp32 products and sums must not be contracted into fused
multiply-adds, and fp32 division and square root must be correctly rounded.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libob.so")
SOURCES = [os.path.join(CSRC, "kernels.hip"), os.path.join(CSRC, "topk.hip"),
           os.path.join(CSRC, "activation.hip"), os.path.join(CSRC, "linear_grad.hip"),
           os.path.join(CSRC, "embedding.hip"), os.path.join(CSRC, "adamw.hip"),
           os.path.join(CSRC, "linear.hip"), os.path.join(CSRC, "api.cpp")]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3", "-fPIC", "-std=c++17",
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def build(verbose: bool = False) -> str:
    """Compile libob.so next to this file; returns its path.  Always recompiles."""
    def run(args):
        cmd = [hipcc(), *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC, *args]
        if verbose:
            print(" ".join(cmd), flush=True)
        proc = subprocess.run(cmd, capture_output=True, text=True)
        noise = "is not a recognized feature for this target"
        err = "\n".join(l for l in proc.stderr.splitlines() if noise not in l)
        if proc.returncode != 0:
            raise RuntimeError(f"hipcc failed ({proc.returncode}):\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)

    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:   # one compiler a source, in parallel
        names = [os.path.join(objects, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1, 16)) as pool:
            list(pool.map(lambda so: run(["-c", "-o", so[1], so[0]]), zip(SOURCES, names)))
        run(["-shared", "-o", tmp, *names])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
