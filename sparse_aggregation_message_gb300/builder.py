"""Builds libgnnagg.so in-tree from csrc/*.cu for sm_103a with nvcc.

Each translation unit compiles in its own process (in parallel); the shared
library links the CUDA runtime statically.  Rebuilds only when a source or
header is newer than the library."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgnnagg.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# Host code keeps separate multiplies and adds (no contraction into fused
# multiply-adds), so host arithmetic gives the same bits on x86 and Arm.
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-ffp-contract=off",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgnnagg.so")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, extra, build_dir: str = BUILD) -> str:
    obj = os.path.join(build_dir, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(force: bool = False, verbose: bool = False, extra=(), variant: str = "", only=()) -> str:
    """Compile every csrc/*.cu and link libgnnagg.so; returns its path.
    `variant` names a build with extra compile flags kept apart from the
    library (under _build/<variant>/; used by tests of kernel selections);
    `only`: the sources that its flags are for, the others being the
    library's."""
    build_dir = os.path.join(BUILD, variant) if variant else BUILD
    lib = os.path.join(build_dir, "libgnnagg.so") if variant else LIB
    if not force and not _stale(lib):
        return lib
    os.makedirs(build_dir, exist_ok=True)
    srcs = [s for s in _sources() if not only or os.path.basename(s) in only]
    shared = []
    if only:
        names = [os.path.basename(s) for s in _sources() if s not in srcs]
        shared = [os.path.join(BUILD, n + ".o") for n in names]
        if _stale() or not all(map(os.path.exists, shared)):
            build(force=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra), build_dir), srcs)) + shared
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if verbose:
        print("built", lib)
    return lib


if __name__ == "__main__":
    import sys

    build(force="--force" in sys.argv, verbose=True)
