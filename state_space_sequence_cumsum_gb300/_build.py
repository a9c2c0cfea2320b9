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


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) +
            [BINDING, os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(NATIVE)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    common = [nvcc, "-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC, *extra_flags]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = common + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    def compile_binding():
        import torch
        inc = os.path.join(os.path.dirname(torch.__file__), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
        obj = os.path.join(BUILD, "binding.o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-I", sysconfig.get_paths()["include"], "-isystem", inc, "-isystem",
               os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-c", BINDING, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}{r.stderr}")
        return obj, os.path.join(os.path.dirname(torch.__file__), "lib")

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 2)) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, _sources()))
        binding_obj, torch_lib = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, "-shared", *ARCH, "-o", tmp, *objs, "-cudart", "static"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of libssd.so failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)
    # the binding finds libssd.so beside itself and PyTorch's libraries as loaded by torch
    tmp = NATIVE + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, binding_obj, "-L", PKG, "-l:libssd.so", "-L", torch_lib,
                        "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
                        f"-Wl,-rpath,{torch_lib}"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _native.so failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, NATIVE)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
