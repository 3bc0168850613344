"""Build the C-ABI shared library libgemm_f16.so in-tree (``_build/``).

Two translation units compiled side by side (the dense product, and the
ragged products with the router), one ``-gencode`` (sm_103a), shared cudart;
nvcc cross-compiles them on a machine without a GPU.
"""
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libgemm_f16.so")
SOURCES = [os.path.join(CSRC, "gemm_api.cu"), os.path.join(CSRC, "ragged_api.cu")]
DEPS = (SOURCES + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(CSRC, "*.h")))
        + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))))

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-cudart", "shared",
    "-I" + INCLUDE, "-I" + CSRC,
]


def _stale_lib(lib):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in DEPS)


def _compile(lib, extra):
    tmp = lib + ".tmp%d" % os.getpid()
    objects = ["%s.%d.o" % (tmp, i) for i in range(len(SOURCES))]
    try:
        jobs = [subprocess.Popen([NVCC, *FLAGS, *extra, "-c", "-o", o, src]) for o, src in zip(objects, SOURCES)]
        codes = [job.wait() for job in jobs]
        if any(codes):
            raise subprocess.CalledProcessError(next(c for c in codes if c), NVCC)
        subprocess.run([NVCC, *FLAGS, "-shared", "-o", tmp, *objects], check=True)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    os.replace(tmp, lib)
    return lib


def build(force=False, verbose_ptxas=False):
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and not _stale_lib(LIB):
        return LIB
    return _compile(LIB, ["-Xptxas", "-v"] if verbose_ptxas else [])


# The measurement build with phase stamps in the single-CTA / CTA-pair kernel
# (GEMM_F16_PHASE_TRACE; see gemm_f16_trace_set).  Never loaded by the product.
TRACE_LIB = os.path.join(OUT_DIR, "libgemm_f16_trace.so")


def build_trace(force=False):
    os.makedirs(OUT_DIR, exist_ok=True)
    if not force and not _stale_lib(TRACE_LIB):
        return TRACE_LIB
    return _compile(TRACE_LIB, ["-DGEMM_F16_PHASE_TRACE"])


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
