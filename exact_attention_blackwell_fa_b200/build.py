"""Compile the CUDA library libfa.so in-tree for sm_100a (nvcc, no GPU needed)."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfa.so")
ROOT = os.path.dirname(HERE)

# each source with the files it includes
SOURCES = {
    "fa_api.cu": ["fa_host.h", "fa_fwd.cuh", "fa_bwd.cuh", "fa_bwd_wide.cuh", "fa_common.cuh", "sm100.cuh",
                  "exp2_poly.h"],
    "fa_paged.cu": ["fa_host.h", "fa_paged.cuh", "fa_paged_fwd.cuh", "sm100.cuh"],
}
OBJ = os.path.join(CSRC, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v"]


def _deps(src: str) -> list:
    return [os.path.join(CSRC, f) for f in (src, *SOURCES[src])] + [os.path.join(ROOT, "include", "fa.h")]


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def _stale() -> bool:
    return any(_older(LIB, _deps(src)) for src in SOURCES)


def _run(cmd) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed to build libfa.so")
    return res.stderr


def _compile(src: str, force: bool) -> tuple:
    """The object file of one source, compiled if it is missing or older than what it is made from."""
    obj = os.path.join(OBJ, src + ".o")
    if not force and not _older(obj, _deps(src)):
        return obj, ""
    tmp = obj + f".tmp{os.getpid()}"
    log = _run([os.environ.get("NVCC", "nvcc"), *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", tmp])
    os.replace(tmp, obj)
    return obj, log


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libfa.so next to this file if it is missing or older than its sources (the sources in parallel)."""
    if not force and not _stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(len(SOURCES)) as pool:
        done = list(pool.map(lambda src: _compile(src, force), SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([os.environ.get("NVCC", "nvcc"), *ARCH, "-shared", "-o", tmp, *[obj for obj, _ in done]])
    if verbose:
        sys.stderr.write("".join(log for _, log in done))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
