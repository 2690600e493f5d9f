"""Builds libstreamkl.so and _calls.so in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each ``csrc/*.cu`` file is compiled in parallel to ``_build/*.o`` and the
objects are linked into ``libstreamkl.so`` beside this file; the library knows
nothing of Python or PyTorch.  ``csrc/calls.cpp``, the package's own caller of
the per-layer entry points, becomes ``_calls.so``, which loads the library
beside it.  Objects are rebuilt when their source, any header, or this script
is newer, and ``_calls.so`` when PyTorch is.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libstreamkl.so")
CALLS = os.path.join(HERE, "_calls.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.path.join(os.environ.get("CUDA_HOME", ""), "bin", "nvcc"), shutil.which("nvcc") or "",
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set CUDA_HOME or put nvcc on PATH)")


def _newest(paths) -> float:
    return max((os.path.getmtime(p) for p in paths), default=0.0)


def _torch():
    """PyTorch's folder, the flags that compile against its headers, and when it was installed."""
    import torch
    root = os.path.dirname(torch.__file__)
    include = os.path.join(root, "include")
    flags = ["-O2", "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"), "-I",
             sysconfig.get_paths()["include"], f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    return root, flags, os.path.getmtime(os.path.join(root, "version.py"))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link; returns the path of libstreamkl.so."""
    os.makedirs(BUILD, exist_ok=True)
    calls = os.path.join(CSRC, "calls.cpp")
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu"))) + [calls]
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    dep_time = _newest(headers)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    torch_dir, torch_flags, torch_time = _torch()

    def compile_one(src: str):
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        newest = max(os.path.getmtime(src), dep_time, torch_time if src == calls else 0.0)
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
            return obj, ""
        cmd = [cc, *ARCH, *CFLAGS, *(torch_flags if src == calls else extra), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max(1, len(sources))) as ex:
        results = list(ex.map(compile_one, sources))
    *objs, calls_obj = [o for o, _ in results]
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                sys.stdout.write(log)
    libs = os.path.join(torch_dir, "lib")
    for target, parts, flags in (
            (LIB, objs, []),
            (CALLS, [calls_obj], [f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-L{HERE}",
                                  "-l:libstreamkl.so", "-Xlinker", "-rpath", "-Xlinker", "$ORIGIN"])):
        if force or not os.path.exists(target) or os.path.getmtime(target) < _newest(parts):
            tmp = target + ".tmp"
            r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *parts, *flags], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, target)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
