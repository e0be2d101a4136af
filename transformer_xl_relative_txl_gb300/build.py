"""Builds the in-tree shared library libtxl_relattn.so for sm_103a, and the
extension module _paged.so that hands torch tensors to it.

Each CUDA translation unit under csrc/ is compiled in parallel with nvcc to an
object in _build/, then nvcc links the shared library next to this file.  The
module is one host file compiled beside them against the headers of Python and
of the installed PyTorch.  No cmake; a few seconds per unit.  Run ``python transformer_xl_relative_txl_gb300/build.py``
(it does not import the package, which needs the library).
"""

from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtxl_relattn.so")
BINDING = os.path.join(PKG, "_paged.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
    return obj, res.stderr


def _compile_binding():
    nvcc = os.path.realpath(_nvcc())
    # found without importing torch, which takes longer than the compiler
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include = [sysconfig.get_paths()["include"], os.path.join(torch, "include"),
               os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"), INCLUDE]
    obj = os.path.join(BUILD, "paged_binding.o")
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           *[f"-I{d}" for d in include], "-c", os.path.join(CSRC, "paged_binding.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for paged_binding.cpp:\n{res.stdout}\n{res.stderr}")
    return obj, os.path.join(torch, "lib")


def _link(cmd, target):
    tmp = target + ".tmp"
    res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, target)


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, list(extra)), srcs))
    objs = [o for o, _ in results]
    if verbose:
        for _, err in results:
            if err.strip():
                print(err, file=sys.stderr)
    _link([_nvcc(), *ARCH, "-shared", *objs], LIB)
    # Behind the library, which every other call needs and this one's headers are not part of.
    obj, torch_lib = binding.result()
    _link([shutil.which("g++") or "c++", "-shared", obj, f"-L{PKG}", "-l:libtxl_relattn.so", f"-L{torch_lib}",
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], BINDING)
    return LIB


if __name__ == "__main__":
    verbose = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if verbose else []
    print(build(verbose=verbose, extra=extra))
