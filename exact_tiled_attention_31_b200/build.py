"""Build the sm_100a shared library ``libfa.so`` in-tree with nvcc.

``python -m exact_tiled_attention_31_b200.build`` (or ``build_library()``)
compiles ``csrc/fa_api.cu`` and ``csrc/fa_paged.cu`` (which include the
kernels) for ``arch=compute_100a, code=sm_100a`` and links the CUDA runtime statically, so
the library loads on a machine without a GPU (for the export checks) and
needs no JIT cache on the machine that runs it.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libfa.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the sm_100a library cannot be built")


UNITS = ("fa_api.cu", "fa_paged.cu")  # translation units of the library


def _needs(path: str, seen=None) -> set:
    """``path`` and every file it includes by a quoted name."""
    seen = set() if seen is None else seen
    path = os.path.normpath(path)
    if path not in seen:
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), flags=re.M):
                _needs(os.path.join(os.path.dirname(path), name), seen)
    return seen


def _newer(target: str, sources) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(s) <= os.path.getmtime(target) for s in sources)


def up_to_date(lib: str = LIB) -> bool:
    return _newer(lib, set().union(*(_needs(os.path.join(CSRC, u)) for u in UNITS)))


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile libfa.so if it is missing or older than its sources; return its
    path.  Units whose object is up to date are not compiled again; the others
    are compiled side by side."""
    if not force and up_to_date():
        return LIB
    nvcc, jobs, objs, said = _nvcc(), [], [], []
    for u in UNITS:
        src, obj = os.path.join(CSRC, u), os.path.join(PKG, u[:-3] + ".o")
        objs.append(obj)
        if not force and _newer(obj, _needs(src)):
            continue
        cmd = [nvcc, *ARCH, *FLAGS, "-c", "-I", os.path.join(ROOT, "include"), "-o", obj + ".tmp", src]
        jobs.append((cmd, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = None
    for cmd, obj, job in jobs:
        out = job.communicate()[0]
        said.append(" ".join(cmd) + "\n" + out)
        if job.returncode == 0:
            os.replace(obj + ".tmp", obj)
        else:
            failed = (job.returncode, out)
    if failed is None:
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", LIB + ".tmp", *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        said.append(" ".join(cmd) + "\n" + res.stdout + res.stderr)
        if res.returncode != 0:
            failed = (res.returncode, res.stdout + res.stderr)
    log = os.path.join(PKG, "build.log")
    with open(log, "w") as f:
        f.write("\n".join(said))
    if failed is not None:
        raise RuntimeError(f"nvcc failed ({failed[0]}); see {log}:\n{failed[1][-4000:]}")
    os.replace(LIB + ".tmp", LIB)
    if verbose:
        print("\n".join(said), file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
