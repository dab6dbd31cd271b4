"""Builds libadamas.so in-tree with nvcc for sm_100a (B200).

    python -m token_level_sparse_fwht_b200.build [--verbose]

The library links the CUDA runtime statically, so it shares the process's primary
CUDA context (and torch's streams) without depending on torch's runtime copy.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libadamas.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
         "-Xcompiler", "-fPIC,-O2", "-cudart", "static"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libadamas.so")
    return exe


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def needs_rebuild() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "adamas.h")]
    return any(os.path.getmtime(p) > t for p in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    if not force and not needs_rebuild():
        return LIB
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objs:
        # one compiler per source file, side by side
        jobs = []
        for src in sources():
            obj = os.path.join(objs, os.path.basename(src)[:-3] + ".o")
            cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
                print(" ".join(cmd))
            jobs.append((obj, cmd))
        with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
            for ok in pool.map(lambda job: _run(job[1], verbose), jobs):
                if not ok:
                    raise RuntimeError("nvcc failed building libadamas.so")
        if not _run([nvcc(), *ARCH, "-cudart", "static", "-shared", *(o for o, _ in jobs), "-o", tmp],
                    verbose):
            raise RuntimeError("nvcc failed linking libadamas.so")
    os.replace(tmp, LIB)
    return LIB


def _run(cmd, verbose: bool) -> bool:
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    elif verbose:
        sys.stdout.write(res.stdout + res.stderr)
    return res.returncode == 0


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(LIB)
