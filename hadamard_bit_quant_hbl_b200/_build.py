"""Build the CUDA library libhbl.so in-tree with nvcc for sm_100a (B200).

Usage: python -m hadamard_bit_quant_hbl_b200._build [--verbose] [--changed]
(--changed: only what is older than its sources)
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libhbl.so")
OBJ = os.path.join(PKG, "build")  # object files, one per .cu

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhbl.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")))


def _deps(path: str, seen: set[str] | None = None) -> set[str]:
    """The file and every header of this repository that it includes."""
    seen = set() if seen is None else seen
    if path not in seen:
        seen.add(path)
        with open(path, encoding="utf-8") as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M):
                for d in (CSRC, INCLUDE):
                    if os.path.exists(os.path.join(d, name)):
                        _deps(os.path.join(d, name), seen)
    return seen


def _newer(target: str, deps) -> bool:
    """Whether target exists and is no older than any of deps."""
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, sources() + [os.path.join(INCLUDE, "hbl.h"), os.path.abspath(__file__)])


def _run(cmd: list[str]) -> str:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return res.stdout + res.stderr


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile the .cu files of csrc (in parallel; each includes its kernels) and link them into
    libhbl.so; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        if force or not _newer(obj, _deps(src) | {os.path.abspath(__file__)}):
            cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj + ".tmp"]
            out = _run(cmd + (["-Xptxas", "-v"] if verbose else []))
            if verbose:
                sys.stdout.write(out)
            os.replace(obj + ".tmp", obj)
        return obj

    with ThreadPoolExecutor() as pool:
        objs = list(pool.map(compile_one, [f for f in sources() if f.endswith(".cu")]))
    tmp = LIB + ".tmp"
    _run([_nvcc(), *NVCC_FLAGS, "-shared", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force="--changed" not in sys.argv)
    print(LIB)
