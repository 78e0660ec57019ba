"""Build the CUDA library ``libssd_gb300.so`` in-tree with nvcc (sm_103a), and
the Python extension ``_ssd_binding.*.so`` with g++.

Each ``csrc/*.cu`` compiles to an object in parallel, then one ``nvcc
-shared`` link.  ``csrc/binding.cpp`` compiles against Python's and torch's
headers, for the calls of ``selective.py`` alone: the library builds and loads
without it.  Outputs go to ``_build/`` beside this file (git-ignored).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libssd_gb300.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libssd_gb300.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(INCLUDE, "ssd.h"), os.path.abspath(__file__)]


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def binding_path() -> str:
    """The Python extension of this torch and this interpreter: it holds to the layout of both."""
    import torch
    return os.path.join(BUILD, f"_ssd_binding.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")


def build_binding(force: bool = False) -> str:
    """Builds the Python extension if its source is newer; returns its path."""
    path = binding_path()
    if not force and _newer(path, [BINDING_SRC, os.path.join(INCLUDE, "ssd.h"), os.path.abspath(__file__)]):
        return path
    import torch
    os.makedirs(BUILD, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    tmp = path + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{INCLUDE}", f"-I{os.path.join(root, 'include')}",
           f"-I{os.path.join(root, 'include', 'torch', 'csrc', 'api', 'include')}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{os.path.join(os.path.dirname(_nvcc()), '..', 'include')}",
           BINDING_SRC, "-o", tmp, f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    objdir = os.path.join(BUILD, "obj")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True), build_binding(force=True))
