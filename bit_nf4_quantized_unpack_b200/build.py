"""Build the C-ABI library ``lib/libqlora.so`` from ``csrc/`` with nvcc for sm_100a.

The Python calls of the microscaled 4-bit operators go through a second, small library,
``lib/qlora_binding.so`` (g++, torch's headers), which loads the first. Where torch or the headers
are not installed the C library is built alone (``python bit_nf4_quantized_unpack_b200/build.py``).

Run ``python -m bit_nf4_quantized_unpack_b200.build`` (or call ``build()``). Objects go
to ``_build/`` at the repository root; the library is written in-tree next to this
file so that it ships with a snapshot of the repository.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "lib", "libqlora.so")
BINDING_SRC = os.path.join(CSRC, "binding", "fp4_binding.cpp")
BINDING = os.path.join(PKG, "lib", "qlora_binding.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-Xptxas", "-v"]
CXX_FLAGS = ["-O2", "-fPIC", "-std=c++17", "-Wall"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _deps_mtime():
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if "." in f] + [os.path.join(INCLUDE, "qlora.h"), __file__]
    return max(os.path.getmtime(p) for p in paths)


def _compile(src, verbose):
    nvcc = _nvcc()
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    if src.endswith(".cu"):
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
    else:
        cmd = ["g++", *CXX_FLAGS, "-I", INCLUDE, "-I", cuda_inc, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr if verbose else ""


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _binding_lacks():
    """What the Python binding cannot be compiled without and is not installed here, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return "torch"
    for path in (os.path.join(os.path.dirname(spec.origin), "include", "torch", "csrc", "utils", "pybind.h"),
                 os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        if not os.path.exists(path):
            return path
    return None


def build_binding(force: bool = False) -> str | None:
    """Compile the Python binding against the running interpreter's torch. Returns its path, or None
    where torch or a header is missing (its calls then raise)."""
    lacks = _binding_lacks()
    if lacks:
        sys.stderr.write(f"{os.path.basename(BINDING)} is left out: no {lacks}\n")
        return None
    import torch
    newest = max(os.path.getmtime(p) for p in (BINDING_SRC, os.path.join(INCLUDE, "qlora.h"), __file__))
    stamp = os.path.join(OBJ, "qlora_binding.torch")  # what the binding was compiled for
    built_for = f"{sys.implementation.cache_tag} torch {torch.__version__}"
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest and _read(stamp) == built_for:
        return BINDING
    root = os.path.dirname(torch.__file__)
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    includes = [os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                cuda_inc, sysconfig.get_paths()["include"]]
    os.makedirs(os.path.dirname(BINDING), exist_ok=True)
    os.makedirs(OBJ, exist_ok=True)
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-fvisibility=hidden",
           f'-DQLORA_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[a for i in includes for a in ("-isystem", i)], BINDING_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
           "-ltorch_python", "-ldl"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(built_for)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every CUDA/C++ source for sm_100a and link the shared library, and the Python
    binding where torch and its headers are installed. Returns the library path. Skips what is
    newer than its sources."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_binding, force)
        path = _build_library(force, verbose)
        binding.result()
    return path


def _build_library(force: bool, verbose: bool) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), sources()))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
