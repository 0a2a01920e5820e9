"""Builds ``libfs.so`` (the CUDA library behind include/fs.h) for sm_100a with nvcc.

The library is built in-tree, next to this file, so that it is the one the Python
binding loads. ``python -m streaming_sinkhorn_b200.build`` rebuilds it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfs.so")
OBJ = os.path.join(HERE, "_build")
SOURCES = ["fs_api.cu", "fs_noalloc.cu", "fs_rows.cu", "fs_linear.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or install the CUDA toolkit)")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files.append(os.path.join(ROOT, "include", "fs.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _object_up_to_date(obj: str, dep: str) -> bool:
    """Whether obj is newer than every file that its last compilation read (nvcc's -MD list)."""
    if not (os.path.exists(obj) and os.path.exists(dep)):
        return False
    t = os.path.getmtime(obj)
    names = open(dep).read().split(":", 1)[1].replace("\\\n", " ").split()
    return all(os.path.exists(f) and os.path.getmtime(f) <= t for f in names)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the sources side by side (only those that changed, unless force) and links."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
             "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
             "--expt-relaxed-constexpr"]
    if verbose:
        flags += ["-Xptxas", "-v"]
    jobs, objects = [], []
    for src in SOURCES:
        obj = os.path.join(OBJ, src + ".o")
        objects.append(obj)
        if not force and _object_up_to_date(obj, obj + ".d"):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc(), *flags, "-MD", "-MF", obj + ".d", "-c", os.path.join(CSRC, src), "-o", tmp]
        jobs.append((subprocess.Popen(cmd), cmd, tmp, obj))
    failed = None
    for proc, cmd, tmp, obj in jobs:
        if proc.wait() != 0:
            failed = failed or subprocess.CalledProcessError(proc.returncode, cmd)
        else:
            os.replace(tmp, obj)
    if failed:
        raise failed
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc(), *ARCH, "-shared", "-o", tmp, *objects], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
