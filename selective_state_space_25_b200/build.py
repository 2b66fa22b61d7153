"""Builds libssmscan.so (the CUDA kernels + C ABI) in-tree with nvcc for
sm_100a.  Run directly (``python -m selective_state_space_25_b200.build``) or
through ``__graft_entry__.build()``.  No GPU is needed to build."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libssmscan.so")
# the debug-bounds build: every kernel checks its global indices (SSM_DEBUG_BOUNDS)
LIB_DEBUG = os.path.join(PKG, "libssmscan_debug.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-Xcompiler", "-Wall"]
# objects, one per source file and build kind (git-ignored)
OBJ_DIR = os.path.join(PKG, "_build")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in deps())


def _closure(path: str, seen=None) -> set:
    """The source and every project header it includes."""
    seen = set() if seen is None else seen
    if path in seen or not os.path.exists(path):
        return seen
    seen.add(path)
    for name in re.findall(r'^#include "([^"]+)"', open(path, encoding="utf-8").read(), flags=re.M):
        for d in (CSRC, INCLUDE):
            _closure(os.path.join(d, name), seen)
    return seen


def _run(cmd, verbose: bool) -> str:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _compile(src: str, force: bool, verbose: bool, ptxas_info: bool, debug_bounds: bool):
    """(object, compiler output) of one source, compiled when it or a header
    it includes is newer than the object."""
    name = os.path.splitext(os.path.basename(src))[0] + ("_debug" if debug_bounds else "")
    obj = os.path.join(OBJ_DIR, name + ".o")
    if not force and os.path.exists(obj) and \
            all(os.path.getmtime(f) <= os.path.getmtime(obj) for f in _closure(src)):
        return obj, ""
    tmp = obj + f".tmp{os.getpid()}.o"
    defs = ["-DSSM_DEBUG_BOUNDS"] if debug_bounds else []
    cmd = [nvcc(), *ARCH, *FLAGS, *defs, f"-I{INCLUDE}", f"-I{CSRC}", "-c", src, "-o", tmp]
    if ptxas_info:
        cmd.insert(1, "-Xptxas=-v")
    out = _run(cmd, verbose)
    os.replace(tmp, obj)
    return obj, out


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          debug_bounds: bool = False) -> str:
    """Builds libssmscan.so, or with debug_bounds libssmscan_debug.so (the
    same sources compiled with SSM_DEBUG_BOUNDS)."""
    lib = LIB_DEBUG if debug_bounds else LIB
    if not force and up_to_date(lib):
        return lib
    os.makedirs(OBJ_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor() as pool:
        done = list(pool.map(lambda s: _compile(s, force, verbose, ptxas_info, debug_bounds),
                             sources()))
    if verbose or ptxas_info:
        sys.stdout.write("".join(out for _, out in done))
    tmp = lib + f".tmp{os.getpid()}"
    _run([nvcc(), *ARCH, "-shared", *(obj for obj, _ in done), "-o", tmp], verbose)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    for dbg in (False, True):
        print("built", build(force="--force" in sys.argv, verbose=True,
                             ptxas_info="--ptxas-info" in sys.argv, debug_bounds=dbg))
