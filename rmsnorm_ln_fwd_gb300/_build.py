"""Build libnorm.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and
_bind.so (the Python binding of the residual-stream operators) with g++ against
the installed PyTorch.

Each .cu translation unit is compiled in parallel, then linked into a shared
library with the CUDA runtime linked statically; the binding links to it.  Both
are rebuilt only when a source or header is newer, when they were built for
another CPU architecture (the GPU hosts are aarch64), or, the binding, for
another PyTorch.
"""

from __future__ import annotations

import glob
import os
import platform
import re
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libnorm.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC] + ARCH

_ELF_MACHINE = {"x86_64": 62, "aarch64": 183, "arm64": 183}


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libnorm.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _elf_machine(path):
    try:
        with open(path, "rb") as f:
            head = f.read(20)
        if head[:4] != b"\x7fELF":
            return None
        return int.from_bytes(head[18:20], "little")
    except OSError:
        return None


def _fresh(lib: str, inputs) -> bool:
    """`lib` exists, for this CPU, and is no older than its inputs."""
    if not os.path.exists(lib):
        return False
    want = _ELF_MACHINE.get(platform.machine())
    if want is not None and _elf_machine(lib) != want:
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in inputs)


def up_to_date(lib: str = LIB) -> bool:
    return _fresh(lib, _inputs())


def _bind_inputs():
    return [BIND_SRC, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))


def bind_torch():
    """The PyTorch version _bind.so was compiled for, read from the file (to load
    it beside another one is undefined); None without one."""
    try:
        with open(BIND, "rb") as f:
            m = re.search(rb"norm_bind_torch=([^\0]+)\0", f.read())
    except OSError:
        return None
    return m.group(1).decode() if m else None


def bind_up_to_date() -> bool:
    import torch
    return bind_torch() == str(torch.__version__) and _fresh(BIND, _bind_inputs())


def _compile_bind() -> str:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), "/usr/local/cuda/include", sysconfig.get_paths()["include"]]
    obj = os.path.join(BUILD_DIR, "bind.cpp.o")
    cmd = [os.environ.get("CXX", "g++"), "-c", BIND_SRC, "-o", obj, "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DNORM_BIND_TORCH="{torch.__version__}"']
    for i in include:
        cmd += ["-isystem", i]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{p.stdout}\n{p.stderr}")
    return obj


def _link_bind(obj: str) -> None:
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB, "-L", tlib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{tlib}"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link of the Python binding failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, BIND)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every CUDA source for sm_103a, link libnorm.so and the Python
    binding; return the library's path."""
    bind = force or not bind_up_to_date()
    if not force and not extra_flags and up_to_date():
        if bind:
            os.makedirs(BUILD_DIR, exist_ok=True)
            _link_bind(_compile_bind())
        return LIB
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags) + (["-Xptxas", "-v"] if verbose else [])

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, "-c", src, "-o", obj] + flags
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{p.stdout}\n{p.stderr}")
        return obj, p.stdout + p.stderr

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources()) + 1, os.cpu_count() or 1))) as ex:
        bind_obj = ex.submit(_compile_bind) if bind else None
        results = list(ex.map(compile_one, sources()))
        bind_obj = bind_obj.result() if bind else None
    tmp = LIB + ".tmp"
    # -ldl: the header-only NVTX ranges look their tool up with dlopen
    cmd = [nvcc, "-shared", "-Xlinker", "-soname=libnorm.so", "-o", tmp] + [o for o, _ in results] + ARCH + ["-cudart", "static", "-ldl"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, LIB)
    if bind:
        _link_bind(bind_obj)
    if verbose:
        for _, log in results:
            print(log)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
