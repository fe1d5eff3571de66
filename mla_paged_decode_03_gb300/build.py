"""Builds libmla_decode.so in-tree (``mla_paged_decode_03_gb300/lib/``) with nvcc for
sm_103a.  Each translation unit compiles in parallel; the CUDA runtime is linked
statically so the library needs only the driver at run time.  Beside it q8_binding.so, the
Python binding of the 8-bit cache's calls, host code against PyTorch's headers; the library
is there without it."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
OBJDIR = os.path.join(LIBDIR, "obj")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIBNAME = "libmla_decode.so"
BINDING = "q8_binding"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    cand = [os.environ.get("NVCC", ""), shutil.which("nvcc") or "", "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def lib_path() -> str:
    return os.path.join(LIBDIR, LIBNAME)


def _compile(src: str, extra) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def binding_path() -> str:
    return os.path.join(LIBDIR, BINDING + ".so")


def _build_binding() -> str:
    """Compiles the binding; returns its path until it takes its place beside the library."""
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    tmp = binding_path() + ".tmp"
    # (symbols of libtorch come from the process that imports it)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *("-I" + d for d in (INCLUDE, CSRC, os.path.join(home, "include"),
                                os.path.join(home, "include", "torch", "csrc", "api", "include"),
                                sysconfig.get_path("include"),
                                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"))),
           os.path.join(CSRC, BINDING + ".cpp"), "-o", tmp, "-L" + os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{BINDING} failed:\n{r.stdout}\n{r.stderr}")
    return tmp


def build(verbose: bool = False, extra=None) -> str:
    extra = list(extra or [])
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    out = lib_path()
    tmp = out + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    if verbose:
        print("built", out)
    # the library stands; a binding that does not compile leaves no older one beside it
    try:
        os.replace(binding.result(), binding_path())
    except BaseException:
        if os.path.exists(binding_path()):
            os.remove(binding_path())
        raise
    return out


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
