"""Build libpisa.so (the CUDA library behind the C ABI in include/pisa.h).

    python -m block_sparse_attention_stats_b200.build [--verbose-ptxas]

Compiles each translation unit csrc/*.cu for sm_100a with nvcc, side by side,
and links libpisa.so next to this file (in-tree, so it travels with the
repository snapshot).  Rebuilds only when a source or header is newer than the
library, unless force=True.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libpisa.so")
OBJ = os.path.join(PKG, "_build")   # objects of one run, removed after the link

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    if os.path.exists(cand):
        return cand
    p = shutil.which("nvcc")
    if not p:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return p


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, ptxas_verbose: bool = False, log: str = "") -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = [*ARCH_FLAGS, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
             "-cudart", "static", "-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stderr

    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(OBJ, f"{os.path.basename(u)}.{os.getpid()}.o") for u in units]
    try:
        with concurrent.futures.ThreadPoolExecutor(len(units)) as pool:
            said = "".join(pool.map(lambda uo: run([_nvcc(), *flags, "-c", "-o", uo[1], uo[0]]),
                                    zip(units, objs)))
        run([_nvcc(), *ARCH_FLAGS, "--shared", "-Xcompiler", "-fPIC", "-cudart", "static",
             "-o", LIB + ".tmp", *objs])
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
    if ptxas_verbose:
        if log:
            with open(log, "w") as f:
                f.write(said)
        else:
            sys.stderr.write(said)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
