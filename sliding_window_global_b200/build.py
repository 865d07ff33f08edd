"""Build libswa.so in-tree with nvcc for sm_100a (no JIT cache, no pip install)."""
from __future__ import annotations

import concurrent.futures
import glob
import hashlib
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libswa.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "-cudart", "shared",
    "-Xlinker", "-rpath,/usr/local/cuda/lib64",
]
LINK_FLAGS = FLAGS[-2:]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in sources() + headers())


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not needs_build():
        return LIB
    # one nvcc per source, side by side; objects newer than their source and every
    # header are kept, those of a build with extra flags in a folder of their own
    objdir = os.path.join(HERE, "_build")
    if extra:
        objdir = os.path.join(objdir, hashlib.sha256("\0".join(extra).encode()).hexdigest()[:16])
    os.makedirs(objdir, exist_ok=True)
    hdr = max(os.path.getmtime(f) for f in headers() + [os.path.abspath(__file__)])
    flags = [f for f in FLAGS if f not in LINK_FLAGS]
    jobs, objs = [], []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or extra or not os.path.exists(obj) or os.path.getmtime(obj) <= max(os.path.getmtime(src), hdr):
            jobs.append(([NVCC, *flags, *extra, "-I", INCLUDE, "-c", "-o", obj + ".tmp", src], obj))
    with concurrent.futures.ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as pool:
        list(pool.map(lambda j: _run(j[0], j[1], verbose), jobs))
    _run([NVCC, *FLAGS, "-shared", "-o", LIB + ".tmp", *objs], LIB, verbose)
    return LIB


def _run(cmd, out, verbose):
    """Run one nvcc command that writes ``out`` + ".tmp", then put the file in place."""
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
