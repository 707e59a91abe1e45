"""Build libmoe.so (the C ABI of include/moe.h) in-tree with nvcc for sm_103a.

Each .cu file compiles to an object in parallel, then one shared library is
linked with the CUDA runtime static, so the library loads without a driver
(the symbol-export check runs on machines without a GPU).  Beside it the module
_binding.so (csrc/binding.cpp), which takes the dense operators' arguments from
Python, linked against the library and the torch that is installed."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIB_DIR, "libmoe.so")
BINDING = os.path.join(LIB_DIR, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _inputs():
    """The library's sources, what they depend on, and what the binding does."""
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    both = [os.path.join(ROOT, "include", "moe.h"), __file__]
    return srcs, srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + both, \
        [os.path.join(CSRC, "binding.cpp"), *both]


def _current(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    _, lib_deps, binding_deps = _inputs()
    return _current(LIB, lib_deps) and _current(BINDING, binding_deps)


def _binding_command(src: str, obj: str):
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
            "-isystem", sysconfig.get_paths()["include"], "-c", src, "-o", obj]


def _link_binding(obj: str):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    _run([shutil.which("g++") or "g++", "-shared", "-o", tmp, obj, "-L", LIB_DIR, "-l:libmoe.so", "-L", libs, "-ltorch_python", "-ltorch_cpu",
          "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs], "link failed")
    os.replace(tmp, BINDING)


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    """Builds what is out of date.  The library needs nvcc alone: where the binding cannot be built (no torch, no
    Python headers) that is raised, with the library in place."""
    srcs, lib_deps, binding_deps = _inputs()
    need_lib, need_binding = force or not _current(LIB, lib_deps), force or not _current(BINDING, binding_deps)
    if not need_lib and not need_binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = _binding_command(src, obj) if src.endswith(".cpp") else [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        return obj, _run(cmd, f"{os.path.basename(cmd[0])} failed on {src}")

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        binding = ex.submit(compile_one, os.path.join(CSRC, "binding.cpp")) if need_binding else None
        results = list(ex.map(compile_one, srcs)) if need_lib else []
    if verbose or ptxas_info:
        for obj, log in results:
            if log.strip():
                print(f"== {os.path.basename(obj)}\n{log}")
    if need_lib:
        tmp = LIB + ".tmp"
        _run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *(o for o, _ in results)], "link failed")
        os.replace(tmp, LIB)
    if need_binding:
        _link_binding(binding.result()[0])
    return LIB


if __name__ == "__main__":
    import sys
    print(build(verbose=True, force="--force" in sys.argv, ptxas_info="--ptxas" in sys.argv))
