"""Build libpagedmla.so (the C-ABI CUDA library) in-tree for sm_103a with nvcc, and the Python
module whose calls turn torch tensors into its descriptors with g++.

The translation units (host API + merge kernels, and one per decode instantiation or
operator) compile in parallel, then link into ``paged_mla_latent_gb300/_build/libpagedmla.so``.
The CUDA runtime is linked statically, so the library loads on a machine without a GPU
(the symbol checks of the CPU test-suite rely on that).  The module is built against the
installed torch, whose version its file name carries; each of the two is rebuilt for its own sources.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libpagedmla.so")
NATIVE_PATH = os.path.join(BUILD_DIR, f"pmla_native.torch{torch.__version__}.so")
NATIVE_SOURCE = os.path.join(CSRC, "native_calls.cpp")
HEADER = os.path.join(os.path.dirname(HERE), "include", "paged_mla.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(CSRC, "*.h")) + [HEADER, os.path.abspath(__file__)])


def native_up_to_date() -> bool:
    return _newer(NATIVE_PATH, [HEADER, NATIVE_SOURCE, os.path.abspath(__file__)])


def up_to_date() -> bool:
    return library_up_to_date() and native_up_to_date()


def _compile(src, obj, verbose=False):
    cmd = [_nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        print(r.stderr)
    return obj


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and library_up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = {src: os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + f".{os.getpid()}.o") for src in _sources()}
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    try:
        with ThreadPoolExecutor(max_workers=len(objs)) as ex:
            list(ex.map(lambda src: _compile(src, objs[src], verbose), objs))
        r = subprocess.run([_nvcc(), *ARCH, "-shared", "-o", tmp, *objs.values()], capture_output=True, text=True)
    finally:
        for o in objs.values():
            try:
                os.remove(o)
            except OSError:
                pass
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _compile_native(obj):
    root = os.path.dirname(torch.__file__)
    include = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in include), "-c", NATIVE_SOURCE, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {NATIVE_SOURCE}:\n{r.stdout}\n{r.stderr}")


def _link_native(obj):
    tmp = NATIVE_PATH + f".tmp{os.getpid()}"
    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-shared", "-o", tmp, obj, f"-L{BUILD_DIR}", "-l:libpagedmla.so", "-Wl,-rpath,$ORIGIN",
           f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    os.remove(obj)
    if r.returncode != 0:
        raise RuntimeError(f"g++ link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Both, at once; the library is in place before a failure of the module's is raised."""
    module = force or not native_up_to_date()
    os.makedirs(BUILD_DIR, exist_ok=True)
    obj = os.path.join(BUILD_DIR, f"native_calls.{os.getpid()}.o")
    with ThreadPoolExecutor(max_workers=1) as ex:
        native = ex.submit(_compile_native, obj) if module else None
        build_library(force, verbose)
    if module:
        native.result()
        _link_native(obj)
    return LIB_PATH


def build_native() -> str:
    """The module alone, next to a library that is there."""
    if not native_up_to_date():
        obj = os.path.join(BUILD_DIR, f"native_calls.{os.getpid()}.o")
        _compile_native(obj)
        _link_native(obj)
    return NATIVE_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
