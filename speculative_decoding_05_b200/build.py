"""Build the CUDA library libdspark.so in-tree for sm_100a (nvcc)."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libdspark.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu (each includes the kernels it launches) into libdspark.so."""
    if not force and not stale():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    with tempfile.TemporaryDirectory(prefix="dspark_build") as tmp:
        jobs, objs = [], []
        for cu in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
            obj = os.path.join(tmp, os.path.basename(cu) + ".o")
            cmd = [nvcc, *NVCC_FLAGS, "-c", "-o", obj, cu]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd), file=sys.stderr)
            jobs.append((cmd, subprocess.Popen(cmd)))
            objs.append(obj)
        codes = [j.wait() for _, j in jobs]
        for (cmd, _), code in zip(jobs, codes):
            if code != 0:
                raise subprocess.CalledProcessError(code, cmd)
        out = LIB + f".tmp{os.getpid()}"
        subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-o", out, *objs], check=True)
        os.replace(out, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
