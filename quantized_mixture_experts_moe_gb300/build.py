"""Builds libqmoe.so (the sm_103a CUDA library) in-tree with nvcc, and _bind.so
(the compiled argument marshalling of the calls around the experts) with g++.

Each .cu file is compiled separately and in parallel, then linked into one
shared library next to this file; _bind.so finds it by its name in its own
folder, so the package can be moved.  Rebuilds only when a source is newer than
the libraries, or _bind.so was built for another Python or torch."""

from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(PKG, "libqmoe.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
BUILD_DIR = os.path.join(PKG, "_build")
STAMP = os.path.join(BUILD_DIR, "bind.txt")  # what _bind.so was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, *ARCH]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + [BIND_SRC] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def bind_target() -> str:
    """The interpreter and the torch whose interfaces _bind.so is compiled against."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"python {sys.version}\ntorch in {_torch_dir()}\n{f.read()}"


def _stamped() -> bool:
    try:
        with open(STAMP) as f:
            return f.read() == bind_target()
    except OSError:
        return False


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND) or not _stamped():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    return all(os.path.getmtime(p) <= t for p in _deps())


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _cuda_include() -> str:
    return os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    def compile_bind():
        obj = os.path.join(BUILD_DIR, "bind.o")
        inc = [sysconfig.get_paths()["include"], os.path.join(_torch_dir(), "include"), _cuda_include()]
        cmd = ["g++", "-O2", "-std=c++20", "-fPIC", *[f"-I{p}" for p in inc], "-c", BIND_SRC, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        bind = ex.submit(compile_bind)
        # the slowest sources first
        order = sorted(sources(), key=os.path.getsize, reverse=True)
        objs = sorted(ex.map(compile_one, order))
        bind_obj = bind.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = BIND + f".tmp{os.getpid()}"
    torch_lib = os.path.join(_torch_dir(), "lib")
    cmd = ["g++", "-shared", "-o", tmp, bind_obj, LIB, "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(STAMP, "w") as f:
        f.write(bind_target())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
