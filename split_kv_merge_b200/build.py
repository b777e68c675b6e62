"""Build libsplitkv.so (sm_100a) in-tree with nvcc.

    python split_kv_merge_b200/build.py [--force]

Each .cu under csrc/ compiles to _build/<name>.o (skipped when newer than its sources and the
headers), then everything links into split_kv_merge_b200/libsplitkv.so with the CUDA runtime
linked statically.  csrc/binding.cpp becomes split_kv_merge_b200/_serving.so, the Python extension of
the serving operators, against torch's libraries and libsplitkv.so (left out where torch is not
installed).  The oracle is pure Python/numpy and needs no build step.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsplitkv.so")
BINDING = os.path.join(PKG, "_serving.so")
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _compile(src: str, force: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    newest = max(os.path.getmtime(p) for p in [src, *_headers(), __file__])
    if force or not os.path.exists(obj) or os.path.getmtime(obj) < newest:
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if "-Xptxas" in extra and r.stderr:
            print(r.stderr, file=sys.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, force, extra), srcs))
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _binding(force)
    return LIB


def _binding(force: bool):
    """The Python extension, made again when its source, the header, torch or the command line changed.  Without torch
    there is none: the library is complete for C callers, and the serving calls say so when they are first used."""
    src = os.path.join(CSRC, "binding.cpp")
    inputs = [src, __file__, os.path.join(ROOT, "include", "splitkv.h")]
    spec = importlib.util.find_spec("torch")
    if spec is None:
        print("torch not found: the Python extension of the serving operators was not built", file=sys.stderr)
        return None
    torch = os.path.dirname(spec.origin)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", src, "-o", BINDING,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"), "-isystem",
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L", PKG, "-lsplitkv", "-Wl,-rpath,$ORIGIN"]  # torch's own libraries are loaded before it
    with open(os.path.join(torch, "version.py")) as f:
        made_with = f"{cmd}\n{f.read()}"
    stamp = os.path.join(BUILD, "serving.made_with")
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= max(map(os.path.getmtime, inputs)):
        if os.path.exists(stamp):
            with open(stamp) as f:
                if f.read() == made_with:
                    return BINDING
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding failed:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made_with)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas-v" in sys.argv))
