"""Builds libvsa.so (the C-ABI library) in-tree with nvcc for sm_103a, and
the paged cache's Python binding beside it with the host compiler.

Each translation unit compiles in its own process (in parallel) and the
CUDA objects link into bwd_tile_mean_gb300/_build/libvsa.so. Objects are
rebuilt when their source or any header is newer; the binding also belongs
to one torch and one Python.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libvsa.so")
SOURCES = ["vsa_api.cu", "index_kernels.cu", "fwd_kernel.cu", "bwd_kernels.cu", "noalloc.cu", "tile3d.cu", "waitcheck.cu",
           "host_step.cu", "check_inputs.cu", "compress_kernels.cu", "paged_append.cu", "paged_select.cu",
           "paged_attn.cu"]
NVCC = os.environ.get("NVCC", "nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose):
    obj = os.path.join(OUT, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(CSRC, src)] + _headers()
    if not _stale(obj, deps):
        return obj
    cmd = [NVCC] + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}")
    return obj


def binding():
    """The paged cache's Python extension for the running Python and the
    installed torch, whose objects it unpacks (dates alone would let the
    binary of an earlier torch pass after a downgrade, or another Python's)."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(OUT, f"paged_binding.torch-{torch.__version__}-abi{abi}.{sysconfig.get_config_var('SOABI')}.so")


def _bind(verbose):
    import torch
    src, target = os.path.join(CSRC, "paged_binding.cpp"), binding()
    if not _stale(target, [src, torch.__file__, os.path.abspath(__file__)] + _headers()):
        return
    at = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    tmp = target + f".{os.getpid()}.tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + INCLUDE, "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(at, "include"),
           "-I" + os.path.join(at, "include", "torch", "csrc", "api", "include"), "-I" + os.path.join(cuda, "include"),
           src, "-o", tmp, "-L" + os.path.join(at, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("the host compiler failed on paged_binding.cpp")
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    if force:
        for o in glob.glob(os.path.join(OUT, "*.o")) + glob.glob(os.path.join(OUT, "paged_binding.*.so")):
            os.remove(o)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_bind, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        binding.result()
    if _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [NVCC] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc link failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
