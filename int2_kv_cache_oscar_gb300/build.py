"""Build liboscar.so (the C-ABI library) in-tree for sm_103a with nvcc.

Each .cu file under csrc/ is compiled in parallel, then linked with the CUDA
runtime statically into int2_kv_cache_oscar_gb300/liboscar.so.  binding.cpp
(the Python calls of the per-step operators, on torch tensors) is compiled
beside them and linked against that library as _calls.so.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liboscar.so")
CALLS = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]
SOURCES = ["quantize.cu", "decode.cu", "prefill.cu", "prefill_tc.cu", "bf16_decode.cu", "rotary.cu", "read.cu",
           "select.cu", "oscar_api.cu"]


def _nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe is None:
        cand = "/usr/local/cuda/bin/nvcc"
        if os.path.exists(cand):
            return cand
        raise RuntimeError("nvcc not found")
    return exe


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _cuda_include() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _compile_binding() -> str:
    import torch
    inc = os.path.join(_torch_dir(), "include")
    obj = os.path.join(BUILD, "binding.o")
    dirs = [sysconfig.get_paths()["include"], inc, os.path.join(inc, "torch", "csrc", "api", "include"), _cuda_include()]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{d}" for d in dirs],
          "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], "g++ of binding.cpp")
    return obj


def _link_binding(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = CALLS + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{PKG}", "-l:liboscar.so", f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
          "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "link of _calls.so")
    os.replace(tmp, CALLS)


def build(verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), SOURCES))
        binding = binding.result()
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
