"""Build the CUDA library libqmv.so in-tree for sm_103a.

Each .cu file is compiled by its own nvcc process (in parallel), then linked
into ``bit_weight_only_packed_gb300/_lib/libqmv.so``.  No fast-math: the
kernels rely on IEEE fp32 rounding.  The binding's host module (C++ against the
running torch's and Python's headers) goes beside it as ``qmv_host.so``, with a note
of what it was built for; the library does without it where it cannot be built.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libqmv.so")
HOST_SRC = os.path.join(CSRC, "host", "qmv_host.cpp")
HOST_LIB = os.path.join(OUT_DIR, "qmv_host.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def cflags(extra=()):
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
            "-I", os.path.join(ROOT, "include"), "-I", CSRC, *extra]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def host_abi() -> str:
    """What the host module's code depends on beside its sources."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def _host_built_for() -> str:
    try:
        with open(HOST_LIB + ".for") as f:
            return f.read()
    except OSError:
        return ""


def build_host(force: bool = False) -> str:
    if not force and _host_built_for() == host_abi() and not _stale(
            HOST_LIB, [HOST_SRC, os.path.join(ROOT, "include", "qmv.h"), __file__]):
        return HOST_LIB
    import torch
    os.makedirs(OUT_DIR, exist_ok=True)
    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    tlib = os.path.join(tdir, "lib")
    inc = [os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
           sysconfig.get_paths()["include"]]
    tmp = HOST_LIB + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-fvisibility=hidden",
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                        *(f for d in inc for f in ("-isystem", d)), "-I", os.path.join(ROOT, "include"), "-o", tmp,
                        HOST_SRC, "-L", tlib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
                        f"-Wl,-rpath,{tlib}"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {HOST_SRC}:\n{r.stderr}")
    if os.path.exists(HOST_LIB + ".for"):       # no note while the module changes
        os.remove(HOST_LIB + ".for")
    os.replace(tmp, HOST_LIB)
    with open(HOST_LIB + ".for", "w") as f:
        f.write(host_abi())
    return HOST_LIB


def _try_host(force: bool = False):
    """The library's calls all work without the host module, so a failure is only told."""
    try:
        build_host(force)
    except (OSError, RuntimeError, AttributeError, ImportError) as e:
        warnings.warn(f"qmv_host.so could not be built: {e}")


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [
        os.path.join(ROOT, "include", "qmv.h"), __file__]
    if not force and not extra and not _stale(LIB, deps):
        _try_host()
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    tmpdir = os.path.join(OUT_DIR, f"obj{os.getpid()}")
    os.makedirs(tmpdir, exist_ok=True)
    cc = nvcc()
    flags = cflags(extra)
    if os.environ.get("QMV_PTXAS_V"):
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(tmpdir, os.path.basename(src) + ".o")
        r = subprocess.run([cc, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        host = ex.submit(_try_host, force)
        objs = list(ex.map(compile_one, sources()))
        host.result()
    tmp_lib = LIB + f".tmp{os.getpid()}"
    link = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp_lib, *objs,
            "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp_lib, LIB)
    shutil.rmtree(tmpdir, ignore_errors=True)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
