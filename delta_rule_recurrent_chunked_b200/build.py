"""Build libdrscan.so in-tree for sm_100a (``python -m delta_rule_recurrent_chunked_b200.build``)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdrscan.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]
# The scans and the operators around them: two units, compiled at the same time.
UNITS = ["drscan.cu", "layer.cu"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in _sources())


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile the units of csrc (which include every kernel) into libdrscan.so."""
    if not force and not needs_build():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = LIB + f".tmp{os.getpid()}"
    objects, running = [], []
    for unit in UNITS:
        objects.append(f"{tmp}.{unit}.o")
        cmd = [nvcc, *NVCC_FLAGS, "-I" + INCLUDE, "-c", "-o", objects[-1],
               os.path.join(CSRC, unit)]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        running.append((cmd, subprocess.Popen(cmd)))
    try:
        codes = [(cmd, p.wait()) for cmd, p in running]
        for cmd, code in codes:
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.check_call([nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *objects])
        os.replace(tmp, LIB)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
