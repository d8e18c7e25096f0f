"""Build libsplitzip.so (the CUDA library behind the C ABI) in-tree for sm_100a,
and _host.*.so (the Python binding's argument checks of the paged-cache operators),
whose name says which Python and torch it is for.

Usage: python fp8_kv_cache_exp_b200/build.py [--force]
(run it by path: importing the package itself loads the library it builds)
"""
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libsplitzip.so")
HOST_SRC = os.path.join(CSRC, "sz_host.cpp")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-O2,-Wall",
    "-Xptxas", "-O3",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(INCLUDE, "splitzip.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def host_path() -> str:
    """The binding's module for this interpreter and its torch, whose tensors it reads by their layout."""
    import sysconfig
    import torch
    return os.path.join(HERE, "_host.torch-%s%s" % (torch.__version__, sysconfig.get_config_var("EXT_SUFFIX")))


def host_up_to_date() -> bool:
    host = host_path()
    return os.path.exists(host) and all(os.path.getmtime(p) <= os.path.getmtime(host)
                                        for p in (HOST_SRC, os.path.join(INCLUDE, "splitzip.h")))


def build_host(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/sz_host.cpp against this interpreter and its torch."""
    host = host_path()
    if not force and host_up_to_date():
        return host
    import sysconfig
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(os.environ.get("NVCC", "nvcc")) or
                                                            "/usr/local/cuda/bin/nvcc")))
    tmp = host + ".tmp.%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", INCLUDE, "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(at, "include"),
           "-isystem", os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-o", tmp, HOST_SRC,
           "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, host)
    return host


def build(force: bool = False, extra_flags=(), out: str = LIB, verbose: bool = False, files=None) -> str:
    """Compile every csrc/*.cu, or the named ones (one nvcc per file, in parallel), and link them
    into one shared library; return its path.  Behind the library itself comes the binding's module,
    which is all that needs torch's headers."""
    if force or out != LIB or not up_to_date():
        build_library(extra_flags, out, verbose, files)
    if out == LIB:
        build_host(force, verbose)
    return out


def build_library(extra_flags, out: str, verbose: bool, files) -> None:
    import tempfile
    from concurrent.futures import ThreadPoolExecutor
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = out + ".tmp.%d" % os.getpid()
    with tempfile.TemporaryDirectory(prefix="splitzip_build_") as objdir:
        def compile_one(src):
            obj = os.path.join(objdir, os.path.basename(src) + ".o")
            cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src]
            if verbose:
                print(" ".join(cmd))
            subprocess.run(cmd, check=True)
            return obj
        srcs = sources() if files is None else [os.path.join(CSRC, f) for f in files]
        with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
            objs = list(ex.map(compile_one, srcs))
        cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
    os.replace(tmp, out)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
