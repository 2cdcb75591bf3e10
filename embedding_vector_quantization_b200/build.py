"""Builds libtq.so in-tree with nvcc for sm_100a (B200).

Usage: ``python embedding_vector_quantization_b200/build.py [--force] [-v]`` (a plain script:
it does not import the package, so a stale library is never loaded first).
The shared library lands next to this file so the Python binding (and any
copy of the repository) finds it without installation.
"""

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtq.so")
SOURCES = ["tq_api.cu", "tq_noalloc.cu", "tq_paged.cu", "host_math.cpp"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _newest_source_mtime():
    newest = 0.0
    for dirpath in (CSRC, os.path.join(ROOT, "include")):
        for name in os.listdir(dirpath):
            if name.endswith((".cu", ".cuh", ".cpp", ".h")):
                newest = max(newest, os.path.getmtime(os.path.join(dirpath, name)))
    return newest


def _stale(obj, dep):
    """Whether an object file is missing or older than a file it was made from (nvcc's dependency file)."""
    if not (os.path.exists(obj) and os.path.exists(dep)):
        return True
    with open(dep) as f:
        names = f.read().replace("\\\n", " ").split(":", 1)[1].split()
    at = os.path.getmtime(obj)
    return any(not os.path.exists(n) or os.path.getmtime(n) > at for n in names)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles libtq.so if missing or older than any source; returns its path.

    Each source has its own object file under _build/, compiled at the same time as the others and only
    when something it includes is newer.
    """
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_source_mtime():
        return LIB
    objs = os.path.join(HERE, "_build")
    os.makedirs(objs, exist_ok=True)
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
             "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    running, made = [], []
    for src in SOURCES:
        obj = os.path.join(objs, src + ".o")
        dep = obj + ".d"
        made.append(obj)
        if not force and not _stale(obj, dep):
            continue
        cmd = [_nvcc(), *flags, "-MD", "-MF", dep, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        if os.path.exists(obj):
            os.remove(obj)
        running.append((cmd, subprocess.Popen(cmd)))
    failed = [cmd for cmd, p in running if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    subprocess.run([_nvcc(), *ARCH, "-shared", *made, "-o", LIB + ".tmp"], check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
