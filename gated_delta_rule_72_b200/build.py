"""Build libgdn.so (the C-ABI library) in-tree with nvcc for sm_100a.

The library is compiled with the CUDA runtime linked statically, so loading
it needs no libcudart on the library path and, until the first CUDA call,
no GPU driver either.
"""
import glob
import hashlib
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libgdn.so")
OBJ = os.path.join(PKG, "_build")      # one object per .cu, rebuilt when a source it includes,
                                       # the flags or the compiler changed

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I" + os.path.join(ROOT, "include"),
]
LINK_FLAGS = NVCC_FLAGS[:2] + ["-shared", "-cudart", "static", "-Xcompiler", "-fPIC"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(ROOT, "include", "gdn.h")])


def _key() -> str:
    """What objects are compiled with besides their sources: the flags and the compiler."""
    try:
        version = subprocess.run([_nvcc(), "--version"], capture_output=True, text=True, check=True).stdout
    except (OSError, subprocess.CalledProcessError):
        return ""                                  # no compiler here: what is built is all there is
    flags = [f for f in NVCC_FLAGS if not f.startswith("-I")] + LINK_FLAGS
    return hashlib.sha256("\n".join(flags + [_nvcc(), version]).encode()).hexdigest()


def _made_with(target: str, key: str) -> bool:
    """`target` was made with this key (or nothing is known of either)."""
    try:
        with open(_key_file(target)) as f:
            return not key or f.read() == key
    except FileNotFoundError:
        return not key


def _key_file(target: str) -> str:
    return os.path.join(OBJ, os.path.basename(target) + ".key")


def _replace(tmp: str, target: str, key: str) -> None:
    """`target` is there with its key, or without one (and then made again)."""
    if os.path.exists(_key_file(target)):
        os.remove(_key_file(target))
    os.replace(tmp, target)
    with open(_key_file(target), "w") as f:
        f.write(key)


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    # (a library that came without its key, say with a copy of the tree, goes by the times alone)
    return all(os.path.getmtime(s) <= t for s in sources()) and \
        (not os.path.exists(_key_file(LIB)) or _made_with(LIB, _key()))


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
    key, tag = _key(), ".tmp%d" % os.getpid()
    objs, running = [], []
    try:
        for src in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
            obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
            objs.append(obj)
            if not force and os.path.exists(obj) and _made_with(obj, key) and \
                    max(_includes(src).values()) <= os.path.getmtime(obj):
                continue
            cmd = [_nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj + tag]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd))
            running.append((obj, cmd, subprocess.Popen(cmd)))
        failed = [(p.returncode, cmd) for _, cmd, p in running if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(*failed[0])
        for obj, _, _ in running:
            _replace(obj + tag, obj, key)
        subprocess.check_call([_nvcc()] + LINK_FLAGS + objs + ["-o", LIB + tag])
        _replace(LIB + tag, LIB, key)
    finally:
        for _, _, p in running:
            p.wait()
        for tmp in [o + tag for o in objs] + [LIB + tag]:
            if os.path.exists(tmp):
                os.remove(tmp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
