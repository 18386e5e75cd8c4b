"""Build libk3mx.so in-tree with nvcc for sm_103a (one -gencode, no cmake).

Each .cu file compiles to its own object in parallel; the objects link into
one shared library next to this file.  Rebuilds only when a source or header
is newer than the library.  csrc/binding.cpp (the host compiler, PyTorch's and
Python's headers) becomes the module that Python calls of k3mx_mx.h go
through, one file per version of the two.  The library does not need it: where
it cannot be compiled, build() warns, and those calls alone raise.
"""
import concurrent.futures
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libk3mx.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def binding_path():
    import torch
    return os.path.join(HERE, f"_k3mx_binding-torch{torch.__version__}-{sys.implementation.cache_tag}.so")


def build_binding(force=False):
    """Compile csrc/binding.cpp; returns the module's path."""
    import torch
    src, out = os.path.join(CSRC, "binding.cpp"), binding_path()
    deps = [src, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if os.path.exists(out):
        if not force and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps):
            return out
        os.remove(out)              # not an older one's calls, should this one not compile
    base = os.path.dirname(os.path.abspath(torch.__file__))
    dirs = [INCLUDE, os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "/usr/local/cuda/include", sysconfig.get_paths()["include"]]
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f for d in dirs for f in ("-isystem", d)], src, "-o", tmp, "-L", os.path.join(base, "lib"),
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def _binding_or_warning(force):
    """None, or why there is no binding."""
    try:
        build_binding(force)
    except Exception as e:                      # (no PyTorch, no headers, no compiler, its errors)
        return f"the Python calls of k3mx_mx.h are not available, their module was not built: {e}"


def build(force=False, verbose_ptxas=False):
    """Compile every kernel source and link libk3mx.so, and the binding's
    module beside it (a warning if that fails); returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_binding_or_warning, force)
        if force or verbose_ptxas or not up_to_date():
            _build_library(verbose_ptxas)
    if binding.result():
        warnings.warn(binding.result())
    return LIB


def _build_library(verbose_ptxas):
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if verbose_ptxas:
        for (_, log), s in zip(results, srcs):
            print(f"== {os.path.basename(s)}\n{log}")
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "shared", "-Xlinker", "-rpath=/usr/local/cuda/lib64",
           "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose_ptxas="-v" in sys.argv))
