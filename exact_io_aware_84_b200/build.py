"""Build libfa.so in-tree with nvcc for sm_100a.

Usage: ``python -m exact_io_aware_84_b200.build [-v]``.  Each ``csrc/*.cu``
is compiled to an object in ``_build/`` (in parallel), then linked into
``exact_io_aware_84_b200/libfa.so``.  Objects are rebuilt when their source
or any header changed.  ``csrc/fa_serve.cpp``, the serving calls' binding to
torch tensors, becomes the module ``exact_io_aware_84_b200/_serve.*.so``, whose
name holds the versions of Python and torch that it was compiled for; without
torch, g++ or Python's headers the build goes on without it.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfa.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc_path() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa.so")
    return p


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, obj: str, verbose: bool, ptxas_v: bool) -> str:
    cmd = [nvcc_path(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return (r.stdout + r.stderr) if (verbose or ptxas_v) else ""


def _build_serve(force: bool = False) -> None:
    """_serve.*.so against the running interpreter's Python and torch headers,
    whose versions are in its name."""
    import sysconfig

    src = os.path.join(CSRC, "fa_serve.cpp")
    newest = max(os.path.getmtime(src), _headers_mtime())
    for old in glob.glob(os.path.join(PKG, "_serve*.so")):   # of any version: none outlives its sources
        if os.path.getmtime(old) < newest:
            os.remove(old)

    import torch

    from . import _serve_path

    so = _serve_path()
    if os.path.exists(so) and not force:
        return
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    dirs = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(home, "include"),
            os.path.join(home, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = f"{so}.{os.getpid()}.tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in dirs), src, "-o", tmp, "-L" + os.path.join(home, "lib"), "-lc10", "-ltorch_cpu",
           "-ltorch_python", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fa_serve.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, so)


def build(verbose: bool = False, force: bool = False, ptxas_v: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_t = _headers_mtime()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        stale = force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_t)
        if stale:
            jobs.append((s, o))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for out in ex.map(lambda so: _compile(so[0], so[1], verbose, ptxas_v), jobs):
            if out:
                print(out, file=sys.stderr)
    if jobs or not os.path.exists(LIB):
        tmp = LIB + ".tmp"
        cmd = [nvcc_path(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    try:
        _build_serve(force)
    except (ImportError, OSError, RuntimeError) as e:   # no torch, no compiler, no headers
        warnings.warn(f"the serving calls' compiled binding was not built, they go through ctypes: {e}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force="-f" in sys.argv, ptxas_v="--ptxas" in sys.argv)
    print(LIB)
