"""Build the sm_100a CUDA library libmoe_b200.so in-tree with nvcc.

    python -m sparse_moe_layer_06_b200.build [--force]

Two translation units (csrc/moe_api.cu: the layer; csrc/ops_api.cu: the
operators around it; each includes its kernel headers) compiled for sm_100a
only, with the CUDA runtime linked statically.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmoe_b200.so")
CSRC = os.path.join(PKG, "csrc")
UNITS = [os.path.join(CSRC, f) for f in ("moe_api.cu", "ops_api.cu")]
OBJ_DIR = os.path.join(ROOT, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-diag-suppress", "177",
]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the sm_100a library cannot be built")
    return cand


def sources(path: str, seen=None) -> set:
    """`path` and every file it includes with quotes, directly or not."""
    seen = set() if seen is None else seen
    path = os.path.normpath(path)
    if path not in seen:
        seen.add(path)
        with open(path) as f:
            for inc in re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M):
                sources(os.path.join(os.path.dirname(path), inc), seen)
    return seen


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _object(unit: str) -> str:
    return os.path.join(OBJ_DIR, os.path.basename(unit) + ".o")


def up_to_date() -> bool:
    return _newer(LIB, set().union(*(sources(u) for u in UNITS)))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    pid = os.getpid()
    running = []
    for unit in UNITS:  # the translation units compile side by side
        obj = _object(unit)
        if not force and _newer(obj, sources(unit)):
            continue
        cmd = [nvcc(), *NVCC_FLAGS, "-c", "-o", f"{obj}.tmp{pid}", unit]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd))
        running.append((obj, subprocess.Popen(cmd)))
    failed = [obj for obj, p in running if p.wait() != 0]
    if failed:
        raise RuntimeError(f"nvcc failed for {', '.join(os.path.basename(o) for o in failed)}")
    for obj, _ in running:
        os.replace(f"{obj}.tmp{pid}", obj)
    tmp = LIB + f".tmp{pid}"
    subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *map(_object, UNITS)], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
