"""Build step for the CUDA library: nvcc, sm_100a, in-tree output.

``python -m selective_state_space_19_b200._build`` (or ``build()``) compiles the
``csrc/*.cu`` files (each includes its kernels), one nvcc process for each, and
links them into ``libs6_b200.so`` next to this file; and ``csrc/s6_torch.cpp``, with
the host compiler and torch's headers, into the Python module ``_s6_torch.so``,
which is linked against that library.  An object file is made again when its own
sources are newer, the module also when torch or Python is another version.
nvcc cross-compiles, so no GPU is needed to build.  The library needs nvcc alone:
it is linked before the module is looked at, and where torch is not installed the
module is left out.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(CSRC, "obj")
LIB = os.path.join(HERE, "libs6_b200.so")
MODULE = os.path.join(HERE, "_s6_torch.so")
CXX = "g++"  # nvcc's host compiler too: the module must share torch's libstdc++, not hold one of its own

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
                  glob.glob(os.path.join(CSRC, "*.cpp")) +
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


def _torch_dir():
    """The directory of the installed torch, or None."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _made_for() -> str:
    """What the module is compiled against: torch's and Python's versions."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return "torch %s, %s" % (version, sys.implementation.cache_tag)


def _module_stamp() -> str:
    """The file, beside the module's object, that says what the module was made for."""
    return os.path.join(OBJ, "s6_torch.made_for")


def _module_current() -> bool:
    try:
        with open(_module_stamp()) as f:
            return f.read() == _made_for()
    except OSError:
        return False


def up_to_date() -> bool:
    if not _fresh(LIB, _sources()):
        return False
    return _torch_dir() is None or (_fresh(MODULE, _sources()) and _module_current())


def _module_flags():
    """Compiler and linker flags for the Python module."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    compile_ = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", *["-I" + d for d in inc]]
    link = ["-shared", "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python", "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
    return compile_, link


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    tag = ".tmp%d.o" % os.getpid()  # (*.o is ignored by git)
    module = _torch_dir() is not None
    if module:
        cxx_flags, cxx_link = _module_flags()
    else:
        print("torch is not installed: %s is not built" % os.path.basename(MODULE), file=sys.stderr)
    jobs, objects = {".cu": [], ".cpp": []}, {".cu": [], ".cpp": []}
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp"))):
        kind = os.path.splitext(src)[1]
        if kind == ".cpp" and not module:
            continue
        obj = os.path.splitext(os.path.join(OBJ, os.path.basename(src)))[0] + ".o"
        objects[kind].append(obj)
        if not force and _fresh(obj, _needs(src)) and (kind == ".cu" or _module_current()):
            continue
        out = ["-c", "-o", obj[:-2] + tag, src]
        cmd = [_nvcc(), *NVCC_FLAGS, "-I" + INCLUDE, *out] if kind == ".cu" else [CXX, *cxx_flags, *out]
        if verbose:
            if kind == ".cu":
                cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        try:
            jobs[kind].append((subprocess.Popen(cmd), obj, cmd))
        except OSError:  # no such compiler: of the module, the library is made all the same
            if kind == ".cu":
                raise
            jobs[kind].append((None, obj, cmd))

    def finish(kind):
        """Waits for one kind's compilers; all of their objects are put in place, or none."""
        failed = [cmd for p, _, cmd in jobs[kind] if p is None or p.wait() != 0]
        for _, obj, _ in jobs[kind]:
            if not failed:
                os.replace(obj[:-2] + tag, obj)
            elif os.path.exists(obj[:-2] + tag):
                os.remove(obj[:-2] + tag)
        return failed

    failed, failed_module = finish(".cu"), finish(".cpp")
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    subprocess.check_call([_nvcc(), *NVCC_FLAGS, "-shared", "-o", LIB + tag, *objects[".cu"]])
    os.replace(LIB + tag, LIB)
    if failed_module:
        raise subprocess.CalledProcessError(1, failed_module[0])
    if module:
        subprocess.check_call([CXX, "-o", MODULE + tag, *objects[".cpp"], *cxx_link])
        os.replace(MODULE + tag, MODULE)
        with open(_module_stamp(), "w") as f:
            f.write(_made_for())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
