"""Builds the CUDA library libswa.so in-tree with nvcc for sm_100a."""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libswa.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-shared",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in deps())


def build(force: bool = False, verbose: bool = False, extra=()) -> str | None:
    srcs = sources()
    if not srcs:
        return None
    if force or stale():
        # every source in its own nvcc process, then the link
        flags = [f for f in NVCC_FLAGS if f != "-shared"]
        with tempfile.TemporaryDirectory() as tmp:
            objs, procs = [], []
            for src in srcs:
                objs.append(os.path.join(tmp, os.path.basename(src) + ".o"))
                cmd = ["nvcc", *flags, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", objs[-1]]
                if verbose:
                    print(" ".join(cmd))
                procs.append((cmd, subprocess.Popen(cmd)))
            failed = [cmd for cmd, proc in procs if proc.wait() != 0]
            if failed:
                raise subprocess.CalledProcessError(1, failed[0])
            subprocess.check_call(["nvcc", *NVCC_FLAGS, "-o", LIB, *objs])
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
