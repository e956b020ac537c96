"""Build libwqmm.so in-tree with nvcc for sm_100a (no JIT cache, no GPU needed), and beside it the compiled torch
binding of the routing and adapter operators, _binding.so."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libwqmm.so")
BINDING = os.path.join(HERE, "_binding.so")  # beside it _binding.so.abi: what it was built for
SOURCES = ["api.cu", "kernels_aux.cu", "kernels_wqmm.cu", "kernels_smallm.cu", "kernels_qmm.cu", "noalloc.cu",
           "route.cu", "kernels_route.cu", "lora.cu", "lora_few.cu", "lora_shrink.cu", "lora_expand.cu",
           "lora_outer.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _older(built: str, inputs) -> bool:
    """Whether `built` is missing or older than one of its inputs."""
    return not os.path.exists(built) or any(os.path.getmtime(f) > os.path.getmtime(built) for f in inputs)


def _inputs(binding: bool) -> list:
    """What the binding, or the library, is built from."""
    own = [f for f in os.listdir(CSRC) if (f == "binding.cpp") == binding]
    return [*(os.path.join(CSRC, f) for f in own), os.path.join(ROOT, "include", "wqmm.h"), __file__]


def _abi() -> str:
    """What a binding is built for: this interpreter and this torch."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__} cxx11abi {torch._C._GLIBCXX_USE_CXX11_ABI}"


def _binding_abi() -> str:
    """What the binding that is there was built for."""
    try:
        with open(BINDING + ".abi") as f:
            return f.read()
    except OSError:
        return ""


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Build what is not up to date.  The library needs nvcc alone; the binding also needs torch, and without it
    there is none."""
    if force or _older(LIB, _inputs(False)):
        build_library(verbose, extra)
    if importlib.util.find_spec("torch") is None:
        print("torch is not installed: no binding of the routing and adapter operators is built", file=sys.stderr)
    elif force or _older(BINDING, _inputs(True)) or _binding_abi() != _abi():
        build_binding(verbose)
    return LIB


def build_library(verbose: bool = False, extra=()) -> str:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    subprocess.run([cc, *ARCH, "-shared", "-Xlinker", "-soname=libwqmm.so", "-o", tmp, *objs, "-Xcompiler", "-fPIC"], check=True)
    os.replace(tmp, LIB)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """Compile csrc/binding.cpp against this interpreter's torch and libwqmm.so beside it."""
    import torch
    from torch.utils import cpp_extension
    include = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
               sysconfig.get_paths()["include"]]
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    # by nvcc, which links the shared C++ runtime that torch's libraries use
    cmd = [nvcc(), *ARCH, "-O2", "-std=c++17", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC,-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f for d in include for f in ("-isystem", d)),
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
           "-lc10_cuda", LIB, "-Xlinker", "-rpath=$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    with open(BINDING + ".abi", "w") as f:
        f.write(_abi())
    return BINDING


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
