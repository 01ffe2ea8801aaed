"""Build libspec.so in-tree for sm_103a (nvcc, one process per translation unit, then link).

Usage: ``python -m mtp_speculative_decoding_spec_gb300.build`` or ``build()`` from Python.
Outputs land next to this file (``_build/`` for objects, ``libspec.so`` for the library); both
are ignored by git. The build runs on any host with nvcc (a GPU is not needed to compile).
"""

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspec.so")
SOURCES = ["gemv.cu", "gemv_tc.cu", "gemv_q4.cu", "gemm_tc.cu", "accept.cu", "commit.cu", "abi.cu",
           "trunk/delta.cu", "trunk/delta_chunk.cu",
           "trunk/attn.cu", "trunk/attn_tc.cu", "trunk/abi.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-v"]


def nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspec.so")
    return path


def _compile(src, verbose):
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    os.makedirs(os.path.dirname(obj), exist_ok=True)
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src),
           "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    # keep ptxas's resource report (registers, spills, shared memory) next to the object
    with open(os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".ptxas.log"), "w") as f:
        f.write(res.stderr)
    return obj, res.stderr if verbose else ""


def _stale(objs):
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(d, f) for top in (CSRC, INCLUDE) for d, _, files in os.walk(top)
            for f in files] + [os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force=False, verbose=False):
    """Compile every CUDA source for sm_103a and link libspec.so. Returns the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if not force and not _stale(None):
        return LIB
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    objs = [r[0] for r in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
