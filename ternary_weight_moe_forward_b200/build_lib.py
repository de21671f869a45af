"""Build libmaple_moe.so (the CUDA library) in-tree for sm_100a.

    python -m ternary_weight_moe_forward_b200.build_lib
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmaple_moe.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fPIC", "-fmad=false", "-Xptxas", "-warn-spills"]


OBJ = os.path.join(PKG, "_build")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps(src):
    """A source file and every file that it includes by a quoted name, transitively."""
    seen, todo = set(), [src]
    while todo:
        f = os.path.realpath(todo.pop())
        if f in seen or not os.path.exists(f):
            continue
        seen.add(f)
        with open(f, encoding="utf-8") as fh:
            todo += [os.path.join(os.path.dirname(f), n) for n in re.findall(r'^\s*#include "([^"]+)"', fh.read(), re.M)]
    return seen


def _stale(out, deps):
    return not os.path.exists(out) or any(os.path.getmtime(d) > os.path.getmtime(out) for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile what is out of date (one object per source, side by side) and link the library."""
    os.makedirs(OBJ, exist_ok=True)
    flags = FLAGS + (["-Xptxas", "-v"] if verbose else [])
    jobs, objs = [], []
    for src in sources():
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, _deps(src)):
            cmd = [NVCC, *flags, "-I", os.path.join(ROOT, "include"), "-c", "-o", obj + ".tmp", src]
            jobs.append((cmd, obj, subprocess.Popen(cmd)))
    failed = [cmd for cmd, _, p in jobs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, obj, _ in jobs:
        os.replace(obj + ".tmp", obj)
    if jobs or _stale(LIB, objs):
        subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC", "-o",
                        LIB + ".tmp", *objs], check=True)
        os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
