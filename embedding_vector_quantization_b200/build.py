"""Builds libtq.so in-tree with nvcc for sm_100a (B200).

Usage: ``python embedding_vector_quantization_b200/build.py [--force] [-v]`` (a plain script:
it does not import the package, so a stale library is never loaded first).
The shared library lands next to this file so the Python binding (and any
copy of the repository) finds it without installation.
"""

import fcntl
import hashlib
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libtq.so")
SOURCES = ["tq_api.cu", "tq_noalloc.cu", "tq_paged.cu", "host_math.cpp"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3", "--expt-relaxed-constexpr"]


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


def _key():
    """What an object depends on besides its files: the compiler's version and the flags (None: there is no compiler)."""
    try:
        version = subprocess.run([_nvcc(), "--version"], check=True, capture_output=True, text=True).stdout
    except (OSError, subprocess.CalledProcessError):
        return None
    return hashlib.sha256("\n".join([version, *ARCH, *FLAGS]).encode()).hexdigest()


def _read(path):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def _stale(src, obj, dep, key):
    """Whether a source's object file is missing, made with other flags, by another compiler or from another copy of the tree, or
    older than a file it was made from (nvcc's dependency file)."""
    if not (os.path.exists(obj) and os.path.exists(dep)) or _read(obj + ".key") != key:
        return True
    names = _read(dep).replace("\\\n", " ").split(":", 1)[1].split()
    at = os.path.getmtime(obj)
    return src not in names or any(not os.path.exists(n) or os.path.getmtime(n) > at for n in names)


def _fresh(key):
    """Whether the library is newer than its sources and, where it came with its record (_build/libtq.key), made as it would be
    here."""
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < _newest_source_mtime():
        return False
    made = _read(os.path.join(HERE, "_build", "libtq.key"))
    return key is None or not made or made == key


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles libtq.so if it is missing, older than any source or made with other flags or another compiler; returns its path.

    Each source has its own object file under _build/, compiled at the same time as the others and only when something it
    includes is newer. One process at a time builds (others wait, and find it done); every file appears under its name
    only when it is whole.
    """
    key = _key()
    if not force and _fresh(key):
        return LIB
    if key is None:
        raise RuntimeError(f"{LIB} is missing or older than its sources, and there is no nvcc to build it")
    objs = os.path.join(HERE, "_build")
    os.makedirs(objs, exist_ok=True)
    with open(os.path.join(objs, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if not force and _fresh(key):
            return LIB
        _compile(objs, key, force, verbose)
    return LIB


def _compile(objs, key, force, verbose):
    flags = [*ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-I", CSRC]
    running, made = [], []
    for src in SOURCES:
        path, obj = os.path.join(CSRC, src), os.path.join(objs, src + ".o")
        made.append(obj)
        if not force and not _stale(path, obj, obj + ".d", key):
            continue
        cmd = [_nvcc(), *flags, "-MD", "-MF", obj + ".d.tmp", "-c", path, "-o", obj + ".tmp"]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), file=sys.stderr)
        running.append((obj, cmd, subprocess.Popen(cmd)))
    failed = []
    for obj, cmd, p in running:
        if p.wait() != 0:
            failed.append(cmd)
            continue
        os.replace(obj + ".d.tmp", obj + ".d")
        os.replace(obj + ".tmp", obj)
        with open(obj + ".key", "w") as f:
            f.write(key)
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    subprocess.run([_nvcc(), *ARCH, "-shared", *made, "-o", LIB + ".tmp"], check=True)
    os.replace(LIB + ".tmp", LIB)
    with open(os.path.join(objs, "libtq.key"), "w") as f:
        f.write(key)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
