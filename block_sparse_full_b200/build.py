"""Build step for libssa.so (the C-ABI library) with nvcc for sm_100a, and for
_marshal.so (argument marshalling for Python, against torch's headers) with g++.

Compiles every ``csrc/*.cu`` to an object under ``_build/`` (in parallel) and
links them into ``block_sparse_full_b200/libssa.so``; ``csrc/marshal.cpp``
becomes ``block_sparse_full_b200/_marshal.so``.  They are rebuilt only when a
source or a header is newer, ``_marshal.so`` also when torch or Python is
another.  Run as ``python -m block_sparse_full_b200.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
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
LIB = os.path.join(PKG, "libssa.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError(f"nvcc not found (tried {cand})")
    return cand


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, obj: str, extra, verbose: bool):
    cmd = [nvcc(), *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _built_for(torch) -> str:
    """The Python and the torch that _marshal.so is compiled against."""
    return f"{sys.implementation.cache_tag} torch {importlib.metadata.version('torch')} {torch.origin}"


def _build_marshal(verbose: bool, force: bool):
    spec = importlib.util.find_spec("torch")
    if spec is None:  # the library stands without it
        print("torch is not installed: _marshal.so is left out", flush=True)
        return
    src = os.path.join(CSRC, "marshal.cpp")
    stamp, key = os.path.join(BUILD, "marshal.txt"), _built_for(spec)
    if not force and not _stale(MARSHAL, [src, os.path.join(INCLUDE, "ssa.h")]) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == key:
                return
    import torch  # only its location and ABI

    t = os.path.dirname(torch.__file__)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), src, "-o", MARSHAL,
           "-L", PKG, "-l:" + os.path.basename(LIB), "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for marshal.cpp:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(key)


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or ptxas_info or _stale(o, [s, *hdrs]):
            jobs.append((s, o))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        futs = {ex.submit(_compile, s, o, extra, verbose): s for s, o in jobs}
        for f in cf.as_completed(futs):
            log = f.result()
            if ptxas_info and log:
                print(f"== {os.path.basename(futs[f])}\n{log}", flush=True)
    if jobs or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libssa.so", "-o", LIB, *objs, "-lcudart_static", "-ldl", "-lrt",
               "-lpthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _build_marshal(verbose, force)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv, force="-f" in sys.argv)
    print(LIB)
