"""Build step for the CUDA library: nvcc, sm_100a, in-tree output.

``python -m selective_state_space_19_b200._build`` (or ``build()``) compiles the
``csrc/*.cu`` files (each includes its kernels), one nvcc process for each, and
links them into ``libs6_b200.so`` next to this file.  An object file is made
again when its own sources are newer.  nvcc cross-compiles, so no GPU is needed
to build.
"""
from __future__ import annotations

import glob
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(CSRC, "obj")
LIB = os.path.join(HERE, "libs6_b200.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _needs(path, seen=None):
    """A source file and the files that it includes, directly or not."""
    seen = set() if seen is None else seen
    if path in seen:
        return seen
    seen.add(path)
    with open(path) as f:
        for name in re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M):
            for at in (CSRC, INCLUDE):
                if os.path.exists(os.path.join(at, name)):
                    _needs(os.path.join(at, name), seen)
    return seen


def _fresh(target, sources) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(s) <= t for s in sources)


def up_to_date() -> bool:
    return _fresh(LIB, _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    tag = ".tmp%d.o" % os.getpid()
    jobs, objects = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objects.append(obj)
        if not force and _fresh(obj, _needs(src)):
            continue
        cmd = [_nvcc(), *NVCC_FLAGS, "-I" + INCLUDE, "-c", "-o", obj[:-2] + tag, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        jobs.append((subprocess.Popen(cmd), obj, cmd))
    failed = [cmd for p, _, cmd in jobs if p.wait() != 0]
    if failed:
        for _, obj, _ in jobs:
            if os.path.exists(obj[:-2] + tag):
                os.remove(obj[:-2] + tag)
        raise subprocess.CalledProcessError(1, failed[0])
    for _, obj, _ in jobs:
        os.replace(obj[:-2] + tag, obj)
    subprocess.check_call([_nvcc(), *NVCC_FLAGS, "-shared", "-o", LIB + tag, *objects])  # (*.o is ignored by git)
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
