"""Build the sm_103a shared library ``libnvfp4moe.so`` in-tree with nvcc.

Each .cu file compiles to an object in parallel, then nvcc links them into one
shared object with the CUDA runtime linked statically, so the library loads on a
machine without a GPU (symbols can be inspected) and needs no torch at all.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libnvfp4moe.so")
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-I" + os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "nvfp4moe.h"),
                                                                  os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def check_launch_registers(source: str, log: str):
    """The 8-bit tile kernels hand registers from some warps to others, and would wait forever for registers that the
    launch did not bring, so the library launches them only as compiled to kLaunchRegs registers. A compiler (see its
    log, ``-Xptxas -v``) or flags that give another count fail here, not at the first call."""
    want = re.search(r"\bkLaunchRegs = (\d+)", source)
    if want is None:
        return
    used = re.findall(r"Compiling entry function '\S*rows_tc_kernelILb1E\S*' for .*?\bUsed (\d+) registers", log, re.S)
    if not used or any(u != want.group(1) for u in used):
        raise RuntimeError("the 8-bit tile kernels have to take %s registers a thread (kLaunchRegs, kEpiRegs and "
                           "kOtherRegs), but were compiled to %s" % (want.group(1), ", ".join(used) or "none"))


def _compile(src: str, extra, verbose: bool = False) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-Xptxas", "-v", *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    with open(src) as f:
        check_launch_registers(f.read(), r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not extra and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra), verbose), srcs))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
