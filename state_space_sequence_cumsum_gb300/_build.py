"""Builds ``libssd.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a,
and ``_native.so`` (the binding of the layer operators) with g++.

Each ``csrc/*.cu`` translation unit is compiled in parallel into
``_build/`` and linked into ``libssd.so`` next to this file.  The CUDA
runtime is linked statically, so loading the library needs no GPU and no
libcuda (the driver is reached at run time through the runtime).
``csrc/binding.cpp`` is compiled beside them against PyTorch's headers and
linked to ``libssd.so``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libssd.so")
NATIVE = os.path.join(PKG, "_native.so")
BINDING = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the SSD library needs the CUDA 13 toolkit")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  _headers())


def binding_up_to_date() -> bool:
    return _newer(NATIVE, [BINDING] + _headers())


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}{r.stderr}")
    return r


def build_library(verbose: bool = False, extra_flags=()) -> str:
    """libssd.so, which needs the CUDA toolkit only."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    common = [nvcc, "-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC, *extra_flags]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        r = _run(common + ["-c", src, "-o", obj], f"nvcc failed for {os.path.basename(src)}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 2)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, "-shared", *ARCH, "-o", tmp, *objs, "-cudart", "static"], "link of libssd.so failed")
    os.replace(tmp, LIB)
    return LIB


def _compile_binding() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, "binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
          os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-c", BINDING, "-o", obj],
         "g++ failed for binding.cpp")
    return obj


def _link_binding(obj) -> str:
    import torch
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    # the binding finds libssd.so beside itself and PyTorch's libraries as loaded by torch
    tmp = NATIVE + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", os.path.dirname(LIB), "-l:libssd.so", "-L", torch_lib,
          "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
          f"-Wl,-rpath,{torch_lib}"], "link of _native.so failed")
    os.replace(tmp, NATIVE)
    return NATIVE


def build_binding() -> str:
    """_native.so, which needs g++, PyTorch's headers and libssd.so."""
    return _link_binding(_compile_binding())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """What is not up to date of both.  What keeps the binding from compiling is
    raised once libssd.so, which does not need it, is there."""
    library, binding = force or not library_up_to_date(), force or not binding_up_to_date()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        if library:
            build_library(verbose, extra_flags)
        if obj:
            _link_binding(obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
