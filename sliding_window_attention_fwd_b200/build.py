"""Builds, in-tree, the CUDA library libswa.so with nvcc for sm_100a and the binding's
extension module (csrc/swa_torch.cpp) with g++."""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import subprocess
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libswa.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
CALLS_SRC = os.path.join(CSRC, "swa_torch.cpp")

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


def torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def torch_version() -> str:
    """The installed torch's version, without importing it."""
    with open(os.path.join(torch_dir(), "version.py")) as f:
        return re.search(r"__version__ *= *['\"]([^'\"]+)", f.read()).group(1)


def calls_path() -> str:
    """The extension module.  It is bound to the torch it was built with, so its file
    bears that version: another torch finds no module instead of a broken one."""
    return os.path.join(HERE, f"_torch_calls-{torch_version()}.so")


def stale() -> bool:
    for built, needs in ((LIB, deps()),
                         (calls_path(), [CALLS_SRC, os.path.join(INCLUDE, "swa.h")])):
        if not os.path.exists(built):
            return True
        if any(os.path.getmtime(p) > os.path.getmtime(built) for p in needs):
            return True
    return False


def calls_command():
    """g++ command of the extension module.  torch and its libraries are loaded
    before it is imported, so it carries no path to them."""
    torch = torch_dir()
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), CALLS_SRC, "-o", calls_path(),
            "-L", os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str | None:
    srcs = sources()
    if not srcs:
        return None
    if force or stale():
        # every source in its own process, then the library's link
        flags = [f for f in NVCC_FLAGS if f != "-shared"]
        with tempfile.TemporaryDirectory() as tmp:
            objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in srcs]
            cmds = [["nvcc", *flags, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
                    for src, obj in zip(srcs, objs)] + [calls_command()]
            if verbose:
                for cmd in cmds:
                    print(" ".join(cmd))
            procs = [(cmd, subprocess.Popen(cmd)) for cmd in cmds]
            failed = [cmd for cmd, proc in procs if proc.wait() != 0]
            if failed:
                raise subprocess.CalledProcessError(1, failed[0])
            subprocess.check_call(["nvcc", *NVCC_FLAGS, "-o", LIB, *objs])
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
