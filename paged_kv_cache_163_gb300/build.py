"""Build libpkv.so in-tree: CUDA kernels for sm_103a plus the C++ block manager,
and _prompt_calls.so, the native argument checks of the Python binding.

Usage: ``python -m paged_kv_cache_163_gb300.build [--force] [--verbose]``.
Translation units compile in parallel; the shared library lands next to this
file.  Objects go to ``_build/`` at the repository root.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpkv.so")
BINDING_SRC = os.path.join(PKG, "binding", "prompt_calls.cpp")
BINDING = os.path.join(PKG, "_prompt_calls.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.isdir(home):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _sources():
    cu = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
    cpp = sorted(f for f in os.listdir(CSRC) if f.endswith(".cpp"))
    hdr = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hdr.append(os.path.join(INCLUDE, "pkv.h"))
    return cu, cpp, hdr


def _stale(obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def _binding_job(cuda):
    """Compile command of _prompt_calls.so; None where torch's or Python's headers are missing."""
    import sysconfig
    python = sysconfig.get_paths()["include"]
    try:
        import torch
    except ImportError:
        return None
    top = os.path.dirname(torch.__file__)
    inc = os.path.join(top, "include")
    if not (os.path.exists(os.path.join(python, "Python.h")) and
            os.path.exists(os.path.join(inc, "torch", "csrc", "autograd", "python_variable.h"))):
        return None
    lib = os.path.join(top, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", python,
            "-isystem", os.path.join(cuda, "include"), BINDING_SRC, "-o", BINDING, "-L", lib, f"-Wl,-rpath,{lib}",
            "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    os.makedirs(BUILD, exist_ok=True)
    cu, cpp, hdr = _sources()
    jobs = []
    objs = []
    for f in cu:
        src = os.path.join(CSRC, f)
        obj = os.path.join(BUILD, f + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdr):
            cmd = [nvcc, ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
            if ptxas_verbose:
                cmd += ["-Xptxas", "-v"]
            jobs.append(cmd)
    for f in cpp:
        src = os.path.join(CSRC, f)
        obj = os.path.join(BUILD, f + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdr):
            jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-I", CSRC,
                         "-I", os.path.join(cuda, "include"), "-c", src, "-o", obj])
    if force or _stale(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "pkv.h")]):
        binding = _binding_job(cuda)
        if binding:
            jobs.insert(0, binding)
        else:
            print("no torch or Python headers: the binding checks its arguments in Python", file=sys.stderr)
    logs = []

    def run(cmd):
        try:
            return _run(cmd, verbose)
        except RuntimeError as e:
            if cmd[-1] != "-lc10":
                raise
            print(f"the binding checks its arguments in Python: {e}", file=sys.stderr)  # its calls do the same without
            return ""
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for out in ex.map(run, jobs):
                logs.append(out)
    if jobs or not os.path.exists(LIB) or _stale(LIB, objs):
        _run([nvcc, ARCH, "-shared", "-o", LIB] + objs + ["-lcudart_static", "-lrt", "-ldl", "-lpthread"],
             verbose)
    if ptxas_verbose:
        print("\n".join(l for l in logs if l.strip()))
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args(argv)
    print(build(a.force, a.verbose, a.ptxas_verbose))


if __name__ == "__main__":
    sys.exit(main())
