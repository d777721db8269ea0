"""Builds libkda.so (the C ABI of include/kda.h) in-tree for sm_100a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libkda.so")
OBJ = os.path.join(HERE, "build")
# Each unit compiles by itself, all at once; its object is kept while nothing that it includes is newer.
UNITS = {
    "kda_lib.cu": ["kda_common.cuh", "kda_decode.cuh", "kda_chunk_simt.cuh", "kda_chunk_tc.cuh", "kda_chunk_2pass.cuh",
                   "kda_bwd_simt.cuh", "kda_bwd_tc.cuh", "tc_ptx.cuh", "tc_tile.cuh", "kda_host.h"],
    "kda_la_lib.cu": ["kda_common.cuh", "kda_la.cuh", "kda_la_simt.cuh", "kda_la_tc.cuh", "kda_la_step.cuh", "kda_launch.cuh",
                      "tc_ptx.cuh", "tc_tile.cuh", "kda_host.h"],
    "kda_norm_lib.cu": ["kda_common.cuh", "kda_launch.cuh", "kda_norm.cuh", "tc_ptx.cuh", "kda_host.h"],
}

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _object(unit: str) -> str:
    return os.path.join(OBJ, unit[:-3] + ".o")


def _newer(target: str, files) -> bool:
    """Is `target` missing or older than one of `files`?"""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in files if os.path.exists(f))


def _sources(unit: str):
    return [os.path.join(HERE, "csrc", f) for f in [unit, *UNITS[unit]]] + [os.path.join(ROOT, "include", "kda.h")]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not _newer(LIB, [f for u in UNITS for f in _sources(u)]):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    cc = nvcc()
    tag = f".tmp{os.getpid()}"
    running = []
    for unit in UNITS:
        if not force and not _newer(_object(unit), _sources(unit)):
            continue
        cmd = [cc, *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", "-o", _object(unit) + tag,
               os.path.join(HERE, "csrc", unit)]
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append((unit, cmd, subprocess.Popen(cmd)))
    codes = [(unit, cmd, p.wait()) for unit, cmd, p in running]
    for unit, cmd, rc in codes:
        if rc:
            raise subprocess.CalledProcessError(rc, cmd)
        os.replace(_object(unit) + tag, _object(unit))
    cmd = [cc, *NVCC_FLAGS[:2], "-shared", "-o", LIB + tag, *[_object(u) for u in UNITS]]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(LIB + tag, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, extra=[a for a in sys.argv[1:] if a != "--force"]))
