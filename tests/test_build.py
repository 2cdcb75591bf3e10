"""When the build script compiles and when not, with a stand-in for nvcc."""

import importlib.util
import os
import shutil
import subprocess
import sys
import time

import pytest

from conftest import ROOT

NVCC = """#!/bin/sh
if [ "$1" = "--version" ]; then cat "$CUDA_HOME/version"; exit 0; fi
echo "$@" >> "$CUDA_HOME/log"
while [ $# -gt 0 ]; do
  case "$1" in -o) out="$2"; shift;; -MF) dep="$2"; shift;; -c) src="$2"; shift;; esac
  shift
done
if [ -n "$src" ]; then
  printf 'half' > "$out"; sleep 0.3; printf 'whole %s' "$src" > "$out"
  printf 'x.o : %s \\\\\\n  %s\\n' "$src" "$(dirname "$src")/common.cuh" > "$dep"
else
  printf 'linked' > "$out"
fi
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    pkg = tmp_path / "repo" / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "repo" / "include").mkdir()
    shutil.copy(os.path.join(ROOT, "embedding_vector_quantization_b200", "build.py"), pkg / "build.py")
    for name in ("tq_api.cu", "tq_noalloc.cu", "tq_paged.cu", "host_math.cpp", "common.cuh"):
        (pkg / "csrc" / name).write_text("//\n")
    (tmp_path / "repo" / "include" / "tq.h").write_text("//\n")
    cuda = tmp_path / "cuda"
    (cuda / "bin").mkdir(parents=True)
    (cuda / "bin" / "nvcc").write_text(NVCC)
    (cuda / "bin" / "nvcc").chmod(0o755)
    (cuda / "version").write_text("one\n")
    monkeypatch.setenv("CUDA_HOME", str(cuda))
    old = time.time() - 100
    for d, _, names in os.walk(tmp_path / "repo"):
        for n in names:
            os.utime(os.path.join(d, n), (old, old))
    return pkg, cuda


def load(pkg):
    spec = importlib.util.spec_from_file_location("_build_script", pkg / "build.py")
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def compiled(cuda):
    """The sources compiled since the last call."""
    log = cuda / "log"
    lines = log.read_text().splitlines() if log.exists() else []
    log.write_text("")
    return sorted(os.path.basename(x.split(" -c ")[1].split()[0]) for x in lines if " -c " in x)


ALL = ["host_math.cpp", "tq_api.cu", "tq_noalloc.cu", "tq_paged.cu"]


def test_builds_what_is_newer(tree):
    pkg, cuda = tree
    b = load(pkg)
    b.build()
    assert compiled(cuda) == ALL
    b.build()
    assert compiled(cuda) == []
    now = time.time() + 5
    os.utime(pkg / "csrc" / "tq_noalloc.cu", (now, now))
    b.build()
    assert compiled(cuda) == ["tq_noalloc.cu"]
    b.build(force=True)
    assert compiled(cuda) == ALL


def test_other_flags_or_another_compiler_build_again(tree):
    pkg, cuda = tree
    b = load(pkg)
    b.build()
    compiled(cuda)
    b.ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
    b.build()
    assert compiled(cuda) == ALL
    b.build()
    assert compiled(cuda) == []
    (cuda / "version").write_text("two\n")
    b.build()
    assert compiled(cuda) == ALL


def test_a_failed_compile_is_not_taken_for_an_object(tree):
    pkg, cuda = tree
    b = load(pkg)
    nvcc = cuda / "bin" / "nvcc"
    nvcc.write_text(NVCC.replace("sleep 0.3;", 'case "$src" in *tq_paged*) exit 1;; esac;'))
    with pytest.raises(subprocess.CalledProcessError):
        b.build()
    assert not os.path.exists(b.LIB)
    compiled(cuda)
    nvcc.write_text(NVCC)
    b.build()
    assert compiled(cuda) == ["tq_paged.cu"]


def test_two_processes_build_once(tree):
    pkg, cuda = tree
    runs = [subprocess.Popen([sys.executable, str(pkg / "build.py")], stdout=subprocess.DEVNULL) for _ in range(3)]
    assert [p.wait() for p in runs] == [0, 0, 0]
    assert compiled(cuda) == ALL
    for name in ALL:
        assert (pkg / "_build" / (name + ".o")).read_text().startswith("whole")


def test_a_copied_tree_compiles_its_own_sources(tree, tmp_path):
    pkg, cuda = tree
    load(pkg).build()
    compiled(cuda)
    shutil.copytree(tmp_path / "repo", tmp_path / "copy")   # objects and their lists of files too
    other = tmp_path / "copy" / "pkg"
    now = time.time() + 5
    os.utime(other / "csrc" / "common.cuh", (now, now))
    load(other).build()
    assert compiled(cuda) == ALL


def test_a_library_that_came_without_its_objects_is_taken(tree):
    pkg, cuda = tree
    b = load(pkg)
    b.build()
    compiled(cuda)
    shutil.rmtree(pkg / "_build")
    b.build()
    assert compiled(cuda) == []


def test_without_a_compiler_a_fresh_library_is_taken(tree, monkeypatch):
    pkg, cuda = tree
    b = load(pkg)
    b.build()
    monkeypatch.setattr(b, "_nvcc", lambda: str(cuda / "nothing"))
    assert b.build() == b.LIB
    now = time.time() + 5
    os.utime(pkg / "csrc" / "common.cuh", (now, now))
    with pytest.raises(RuntimeError, match="nvcc"):
        b.build()
