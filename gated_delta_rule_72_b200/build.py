"""Build libgdn.so (the C-ABI library) in-tree with nvcc for sm_100a.

The library is compiled with the CUDA runtime linked statically, so loading
it needs no libcudart on the library path and, until the first CUDA call,
no GPU driver either.
"""
import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libgdn.so")
OBJ = os.path.join(PKG, "_build")      # one object per .cu, rebuilt when a source it includes changed

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I" + os.path.join(ROOT, "include"),
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "gdn.h")])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def _includes(path, seen=None):
    """`path` and every file it includes by a quoted name, directly or not."""
    seen = {} if seen is None else seen
    path = os.path.normpath(path)
    if path not in seen and os.path.exists(path):
        seen[path] = os.path.getmtime(path)
        with open(path) as f:
            for name in re.findall(r'^\s*#include\s+"([^"]+)"', f.read(), re.M):
                _includes(os.path.join(os.path.dirname(path), name), seen)
    return seen


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    tag = ".tmp%d" % os.getpid()
    objs, running = [], []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if not force and os.path.exists(obj) and max(_includes(src).values()) <= os.path.getmtime(obj):
            continue
        cmd = [_nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj + tag]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd))
        running.append((obj, cmd, subprocess.Popen(cmd)))
    for obj, cmd, p in running:
        if p.wait() != 0:
            raise subprocess.CalledProcessError(p.returncode, cmd)
    for obj, _, _ in running:
        os.replace(obj + tag, obj)
    subprocess.check_call([_nvcc()] + NVCC_FLAGS[:2] + ["-shared", "-cudart", "static", "-Xcompiler", "-fPIC"] + objs + ["-o", LIB + tag])
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
