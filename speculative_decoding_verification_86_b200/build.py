"""Build step: compile the CUDA library ``libspecverify.so`` for sm_100a in-tree.

``python -m speculative_decoding_verification_86_b200.build`` (or
``__graft_entry__.build()``) runs nvcc on the units ``csrc/*.cu``.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspecverify.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
    "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
]


def _nvcc():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "spec_verify.h")])


def build(force: bool = False, verbose: bool = False, extra_flags=(), out: str = LIB) -> str:
    """Build the library unless it is newer than its sources; ``out`` names another file, for a build with
    other ``extra_flags``."""
    newest = max(os.path.getmtime(s) for s in sources())
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest and not extra_flags:
        return out
    tmp = out + ".tmp.%d" % os.getpid()
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objects = ["%s.%s.o" % (tmp, os.path.basename(u)) for u in units]
    cmds = [[_nvcc(), *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-c", u, "-o", o]
            for u, o in zip(units, objects)]
    link = [_nvcc(), *NVCC_FLAGS, "-shared", *objects, "-o", tmp, "-cudart", "static"]
    if verbose:
        for cmd in cmds + [link]:
            print(" ".join(cmd), file=sys.stderr)
    try:
        jobs = [subprocess.Popen(cmd) for cmd in cmds]  # the units compile side by side
        codes = [job.wait() for job in jobs]
        for code, cmd in zip(codes, cmds):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.check_call(link)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
