"""Build libdualqk.so (CUDA, sm_100a) in-tree with nvcc."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdualqk.so")
ROOT = os.path.dirname(HERE)

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xptxas", "-v"]
UNITS = ["dualqk", "rows"]   # translation units, compiled side by side


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "dualqk.h")])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or stale():
        nvcc = os.environ.get("NVCC", "nvcc")
        with tempfile.TemporaryDirectory() as tmp:
            objs = [os.path.join(tmp, u + ".o") for u in UNITS]
            procs = [subprocess.Popen([nvcc, *NVCC_FLAGS, "-c", "-o", o, os.path.join(CSRC, u + ".cu")],
                                      stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                     for u, o in zip(UNITS, objs)]
            logs = [p.communicate()[0] for p in procs]
            link = subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-o", LIB, *objs], capture_output=True, text=True) \
                if not any(p.returncode for p in procs) else None
            if verbose or link is None or link.returncode:
                print("".join(logs) + (link.stdout + link.stderr if link else ""))
            if link is None or link.returncode:
                raise RuntimeError("nvcc failed building libdualqk.so")
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
