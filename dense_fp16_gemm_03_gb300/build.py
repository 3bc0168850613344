"""Build the C-ABI shared library libgemm_f16.so in-tree (``_build/``), and the
Python binding gemm_binding.so that links to it.

Three translation units compiled side by side (the dense product, the ragged
products with the router, and the products with an epilogue), one ``-gencode`` (sm_103a), shared cudart;
nvcc cross-compiles them on a machine without a GPU.  The binding is host code
against PyTorch's and Python's headers; where one of them is missing the library
is built without it.
"""
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libgemm_f16.so")
SOURCES = [os.path.join(CSRC, "gemm_api.cu"), os.path.join(CSRC, "ragged_api.cu"), os.path.join(CSRC, "linear_api.cu")]
BINDING = os.path.join(OUT_DIR, "gemm_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
DEPS = (SOURCES + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(CSRC, "*.h")))
        + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))))

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")
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


def _torch_dir():
    """Where PyTorch is installed, without importing it; None where it is not."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def binding_lacks():
    """What the binding's build needs and does not find here, or None."""
    torch = _torch_dir()
    if not torch:
        return "PyTorch"
    if not shutil.which(CXX):
        return CXX
    needs = [os.path.join(torch, "include", "torch", "csrc", "autograd", "python_variable.h"), os.path.join(torch, "lib", "libtorch_python.so"),
             os.path.join(torch, "lib", "libc10_cuda.so"), os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    return next((f for f in needs if not os.path.exists(f)), None)


def binding_target():
    """The PyTorch and the Python that a binding built here is for: its classes' layouts are theirs."""
    torch, version = _torch_dir(), "none"
    if torch and os.path.exists(os.path.join(torch, "version.py")):
        with open(os.path.join(torch, "version.py")) as f:
            version = next((line.split("=", 1)[1].strip() for line in f if line.startswith("__version__")), "unknown")
    return "PyTorch %s, %s" % (version, sysconfig.get_config_var("SOABI"))


def binding_built_for():
    """What the binding in place was built for (a note beside it), or None."""
    if not (os.path.exists(BINDING) and os.path.exists(BINDING + ".for")):
        return None
    with open(BINDING + ".for") as f:
        return f.read()


def _stale_binding():
    headers = glob.glob(os.path.join(INCLUDE, "*.h"))
    if binding_built_for() != binding_target():
        return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(f) > t for f in [BINDING_SOURCE, *headers])


def _binding_command(torch, out):
    """The compiler's command for the binding's object."""
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE, "-I" + os.path.join(torch, "include"),
            "-I" + sysconfig.get_paths()["include"], "-I" + cuda, "-c", "-o", out, BINDING_SOURCE]


def _link_binding(torch, obj):
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "lib64")
    tmp = BINDING + ".tmp%d" % os.getpid()
    subprocess.run([CXX, "-shared", "-o", tmp, obj, "-L" + OUT_DIR, "-lgemm_f16", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(torch, "lib"),
                    "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", "-L" + cuda, "-lcudart"], check=True)
    os.replace(tmp, BINDING)
    # (the note last: a build for another version that ends between the two is done again)
    with open(tmp, "w") as f:
        f.write(binding_target())
    os.replace(tmp, BINDING + ".for")


def _compile(lib, extra, binding=None):
    """The library, and with `binding` (PyTorch's folder) the binding beside it; the library also where the binding fails."""
    tmp = lib + ".tmp%d" % os.getpid()
    objects = ["%s.%d.o" % (tmp, i) for i in range(len(SOURCES))]
    commands = [[NVCC, *FLAGS, *extra, "-c", "-o", o, src] for o, src in zip(objects, SOURCES)]
    if binding:
        objects.append(tmp + ".binding.o")
        commands.append(_binding_command(binding, objects[-1]))
    try:
        jobs = [subprocess.Popen(c) for c in commands]
        failed = [subprocess.CalledProcessError(code, c) if code else None for c, code in zip(commands, [job.wait() for job in jobs])]
        for error in failed[:len(SOURCES)]:
            if error:
                raise error
        subprocess.run([NVCC, *FLAGS, "-shared", "-o", tmp, *objects[:len(SOURCES)]], check=True)
        os.replace(tmp, lib)
        if binding:
            if failed[-1]:
                raise failed[-1]
            _link_binding(binding, objects[-1])
    finally:
        for o in objects:
            if os.path.exists(o):
                os.remove(o)
    return lib


def build(force=False, verbose_ptxas=False):
    os.makedirs(OUT_DIR, exist_ok=True)
    lacks = binding_lacks()
    torch = None if lacks else _torch_dir()
    if lacks and _stale_binding():
        print("gemm_binding.so is left out: %s is missing (the library needs none of it)" % lacks, file=sys.stderr)
        if os.path.exists(BINDING):
            os.remove(BINDING)
    if force or _stale_lib(LIB):
        return _compile(LIB, ["-Xptxas", "-v"] if verbose_ptxas else [], binding=torch)
    if torch and _stale_binding():
        obj = BINDING + ".tmp%d.o" % os.getpid()
        try:
            subprocess.run(_binding_command(torch, obj), check=True)
            _link_binding(torch, obj)
        finally:
            if os.path.exists(obj):
                os.remove(obj)
    return LIB


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
