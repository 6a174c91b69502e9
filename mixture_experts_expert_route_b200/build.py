"""Builds libmoe_b200.so in-tree with nvcc for sm_100a.

    python -m mixture_experts_expert_route_b200.build [--verbose-ptxas] [--debug-checks]

--debug-checks builds libmoe_b200_debug.so instead: the same library compiled
with MOE_DEBUG_CHECKS, whose kernels validate the permutation they are handed
and report a bad entry in the status word (MOE_ERR_DEVICE).  The binding
loads it when the environment sets MOE_B200_DEBUG_CHECKS=1.  Both build _binding.so too.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SOURCES = ["route_permute.cu", "elementwise.cu", "grouped_gemm.cu", "moe_api.cu", "noalloc.cu",
           "split.cu", "decode.cu", "linear.cu"]
# host code of the CPU/GPU split (g++: the AVX512_BF16 kernel selects its
# instruction set per function and checks the CPU at run time)
HOST_SOURCES = ["host_ffn.cpp"]
HEADERS = ["common.cuh", "kernels.h", "topk.cuh"]
LIB = os.path.join(HERE, "libmoe_b200.so")
BINDING = os.path.join(HERE, "_binding.so")    # a Python extension: moe.linear's call
BINDING_STAMP = os.path.join(ROOT, "_build", "binding.txt")    # what it was built for
LIB_DEBUG = os.path.join(HERE, "libmoe_b200_debug.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def lib_path(debug: bool = False) -> str:
    return LIB_DEBUG if debug else LIB


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HOST_SOURCES + HEADERS]
    deps += [os.path.join(ROOT, "include", h) for h in ("moe.h", "moe_split.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_stamp() -> str:
    """What the extension is built for besides its sources: it uses torch's and Python's own
    object layouts."""
    import torch
    return f"{sys.implementation.cache_tag} torch {torch.__version__} " \
           f"abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def build_binding(force: bool = False) -> None:
    """csrc/binding.cpp against the installed torch (host code only).  The package works
    without it, with slower calls, so a machine without g++ or Python's headers only gets a
    warning."""
    src = os.path.join(CSRC, "binding.cpp")
    deps = (src, os.path.join(ROOT, "include", "moe.h"))
    stamp = _binding_stamp()
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING_STAMP) and \
            open(BINDING_STAMP).read() == stamp and \
            all(os.path.getmtime(BINDING) >= os.path.getmtime(d) for d in deps):
        return
    import torch
    pkg = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    includes = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"],
                os.path.join(pkg, "include"),
                os.path.join(pkg, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include")]
    tmp = BINDING + f".{os.getpid()}.tmp"
    try:
        subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                               "-fvisibility=hidden",
                               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                               *(a for d in includes for a in ("-isystem", d)), src, "-o", tmp,
                               "-L" + os.path.join(pkg, "lib"), "-lc10", "-lc10_cuda",
                               "-ltorch_cpu", "-ltorch_python"])
        os.replace(tmp, BINDING)
        os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
        with open(BINDING_STAMP, "w") as f:
            f.write(stamp)
    except (subprocess.CalledProcessError, OSError) as e:
        warnings.warn(f"{BINDING} was not built ({e}): calls go through ctypes")
        # an extension of other sources, torch or Python must not be taken for this one
        for path in (tmp, BINDING):
            if os.path.exists(path):
                os.remove(path)


def build(force: bool = False, ptxas_verbose: bool = False, debug: bool = False) -> str:
    lib = lib_path(debug)
    build_binding(force and not debug)
    if not force and not _stale(lib):
        return lib
    objdir = os.path.join(ROOT, "_build", "debug" if debug else "release")
    os.makedirs(objdir, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]
    if debug:
        flags += ["-DMOE_DEBUG_CHECKS"]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        subprocess.check_call([nvcc(), *flags, "-c", os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
    for src in HOST_SOURCES:
        obj = os.path.join(objdir, src.replace(".cpp", ".o"))
        subprocess.check_call(["g++", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                               "-pthread", "-I", os.path.join(ROOT, "include"),
                               *(["-DMOE_DEBUG_CHECKS"] if debug else []),
                               "-c", os.path.join(CSRC, src), "-o", obj])
        objs.append(obj)
    tmp = lib + f".{os.getpid()}.tmp"
    subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static",
                           "-Xcompiler", "-pthread"])
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv,
                debug="--debug-checks" in sys.argv))
