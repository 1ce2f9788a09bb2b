"""Build libfibatt.so in-tree with nvcc for sm_103a.

Every translation unit under ``csrc/`` is compiled in parallel into
``_build/`` and linked into ``_build/libfibatt.so`` (CUDA runtime linked
statically, no torch dependency).  A unit is rebuilt when it or any header
under ``csrc/`` or ``include/`` is newer than its object.

``build_library(checks=True)`` builds the same sources with
``-DFIBATT_CHECKS`` into ``_build_checks/libfibatt.so``: the debug library
whose kernels check the bounds of their shared-memory stages, windows and
scratch rows and record a failure in the device error word instead of
making the access.  ``FIBATT_CHECKS=1`` in the environment makes the
binding load it.

``build_binding()`` compiles ``binding/calls.cpp``, the short way from Python into some of
the calls, against this Python and torch into ``_build/_calls.so`` (with the
host compiler; the library itself knows neither).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libfibatt.so")
BINDING = os.path.join(PKG, "binding", "calls.cpp")
CALLS = os.path.join(BUILD, "_calls.so")
BUILD_CHECKS = os.path.join(PKG, "_build_checks")
LIB_CHECKS = os.path.join(BUILD_CHECKS, "libfibatt.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libfibatt needs the CUDA toolkit to build")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _compile(args):
    cmd, obj = args
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {obj}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build_library(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False,
                  checks: bool = False) -> str:
    """Compile and link libfibatt.so (the checks build with checks=True);
    returns its path."""
    build_dir, lib_path = (BUILD_CHECKS, LIB_CHECKS) if checks else (BUILD, LIB)
    flags = NVCC_FLAGS + (["-DFIBATT_CHECKS"] if checks else [])
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    hdr_time = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    jobs, objs = [], []
    for src in _sources():
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        objs.append(obj)
        stale = (force or not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(src)
                 or os.path.getmtime(obj) < hdr_time)
        if stale:
            cmd = [nvcc, *ARCH, *flags, "-I", os.path.join(ROOT, "include"), "-c", src, "-o", obj]
            if ptxas_verbose and src.endswith(".cu"):
                cmd += ["-Xptxas", "-v"]
            jobs.append((cmd, obj))
    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for (cmd, obj), err in zip(jobs, ex.map(_compile, jobs)):
                if verbose and err:
                    print(f"[{os.path.basename(obj)}]\n{err}", file=sys.stderr)
    newest = max(os.path.getmtime(o) for o in objs)
    if force or jobs or not os.path.exists(lib_path) or os.path.getmtime(lib_path) < newest:
        tmp = lib_path + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib_path)
    return lib_path


def build_binding(force: bool = False) -> str:
    """Compile binding/calls.cpp; returns the module's path.  It is built anew
    when it, the header, torch or Python has changed."""
    import sysconfig

    import torch

    home = os.path.dirname(torch.__file__)
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
               os.path.join(ROOT, "include")]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [x for i in include for x in ("-isystem", i)] + [BINDING]
    cmd += ["-L", os.path.join(home, "lib"), f"-Wl,-rpath,{home}/lib", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
            "-ltorch_python"]
    made_with, record = f"{sys.version}\n{torch.__version__}\n{' '.join(cmd)}\n", CALLS + ".txt"
    newest = max(os.path.getmtime(f) for f in (BINDING, os.path.join(ROOT, "include", "fibatt.h")))
    if not force and os.path.exists(CALLS) and os.path.exists(record) and os.path.getmtime(CALLS) >= newest:
        with open(record) as f:
            if f.read() == made_with:
                return CALLS
    os.makedirs(BUILD, exist_ok=True)
    tmp = CALLS + f".tmp{os.getpid()}"
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(record, "w") as f:
        f.write(made_with)
    return CALLS


def build_all(force: bool = False) -> None:
    """The library, its checks build and the binding, compiled side by side."""
    with ThreadPoolExecutor(max_workers=3) as ex:
        jobs = [ex.submit(build_library, force, False, False, c) for c in (False, True)] + [ex.submit(build_binding, force)]
        for f in jobs:
            f.result()


if __name__ == "__main__":
    checks = "--checks" in sys.argv
    print(build_library(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv, checks=checks))
