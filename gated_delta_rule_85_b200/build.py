"""Builds libkda.so (the C ABI of include/kda.h) in-tree for sm_100a with nvcc, and _kda_fast.so, the
Python binding's short way to some of its calls, with the host compiler."""
from __future__ import annotations

import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libkda.so")
FAST = os.path.join(HERE, "_kda_fast.so")
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


def _built_for() -> str:
    """What _kda_fast.so depends on beside its sources."""
    import sys

    import torch

    return f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"


def _fast_stale(sources) -> bool:
    if _newer(FAST, sources):
        return True
    with open(FAST, "rb") as f:
        return _built_for().encode() + b"\0" not in f.read()


def _fast_command(out: str):
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [*ext.include_paths(), sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    return [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DKDA_BUILT_FOR="{_built_for()}"', *[f"-isystem{i}" for i in includes],
            "-o", out, os.path.join(HERE, "csrc", "kda_fast.cpp"), "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            "-L", HERE, "-l:libkda.so", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    fast_sources = [os.path.join(HERE, "csrc", "kda_fast.cpp"), os.path.join(ROOT, "include", "kda.h")]
    stale = force or _newer(LIB, [f for u in UNITS for f in _sources(u)])
    if not stale and not _fast_stale(fast_sources):
        return LIB
    tag = f".tmp{os.getpid()}"

    def run(cmds):
        """All at once: (command, file that it makes)."""
        running = []
        for cmd, _ in cmds:
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append(subprocess.Popen(cmd))
        codes = [p.wait() for p in running]
        for (cmd, target), rc in zip(cmds, codes):
            if rc:
                raise subprocess.CalledProcessError(rc, cmd)
            os.replace(target + tag, target)

    if stale:
        os.makedirs(OBJ, exist_ok=True)
        cc = nvcc()
        run([([cc, *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", "-o", _object(unit) + tag,
               os.path.join(HERE, "csrc", unit)], _object(unit))
             for unit in UNITS if force or _newer(_object(unit), _sources(unit))])
        run([([cc, *NVCC_FLAGS[:2], "-shared", "-Xlinker", "-soname=libkda.so", "-o", LIB + tag,
               *[_object(u) for u in UNITS]], LIB)])
    if force or _fast_stale(fast_sources):
        run([(_fast_command(FAST + tag), FAST)])
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, extra=[a for a in sys.argv[1:] if a != "--force"]))
