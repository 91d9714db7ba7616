"""Compile the CUDA library (libpkv.so) in-tree for sm_103a, and the native
part of the Python binding (pkv_binding.so, host code against torch's headers).

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into one shared library with the CUDA runtime linked statically, so
the library loads on a machine without a GPU driver (calls then fail with a
CUDA error instead of the load failing).
"""
from __future__ import annotations

import importlib.metadata
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
LIB = os.path.join(BUILD, "libpkv.so")
SOURCES = ["api.cu", "plan.cpp", "cache.cpp", "decode.cu", "attn_tc.cu", "merge_append.cu", "attn_static.cu", "swap.cu",
           "ops_api.cu", "tree.cu", "tree_tc.cu", "sparse.cu", "pages.cu"]
HEADERS = ["internal.h", "pool.h", "ptx.cuh", "append.cuh", "merge.cuh", "ops.h", "rows.cuh", "sched.cuh",
           "tc.cuh"]
BINDING = os.path.join(BUILD, "pkv_binding.so")
BINDING_STAMP = os.path.join(BUILD, "pkv_binding.stamp")   # binding_key(), and "built" or "left out"
BINDING_SOURCE = "binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(files, than) -> bool:
    files = list(files) + [os.path.join(ROOT, "include", "pkv.h"), os.path.abspath(__file__)]
    return not os.path.exists(than) or any(os.path.getmtime(f) > os.path.getmtime(than) for f in files)


def _lib_stale() -> bool:
    return _newer((os.path.join(CSRC, s) for s in SOURCES + HEADERS), LIB)


def binding_key() -> str:
    """What the binding is compiled against: the installed torch ("" if there is none) and this interpreter."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return ""
    return f"torch {torch} {sysconfig.get_config_var('EXT_SUFFIX')}"


def built_for():
    """The binding_key() of the last build and whether it made a binding; None before the first."""
    try:
        with open(BINDING_STAMP) as f:
            key, made = f.read().splitlines()
    except (OSError, ValueError):
        return None
    return key, made == "built"


def _binding_stale() -> bool:
    last = built_for()
    if last is None or last[0] != binding_key():
        return True
    return last[1] and _newer([os.path.join(CSRC, BINDING_SOURCE)], BINDING)


def _torch():
    """torch, if there is one with CUDA to compile the binding against."""
    try:
        import torch
    except ImportError:
        return None
    return torch if torch.version.cuda else None


def _compile_binding(torch):
    home = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "binding.o")
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj,
           "-isystem", os.path.join(home, "include"), "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_path("include"), "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           "-I", os.path.join(ROOT, "include"), f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{BINDING_SOURCE} failed (the C library is built):\n{r.stderr}")
    return obj, os.path.join(home, "lib")


def _link_binding(obj, torch_lib):
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", obj, "-o", tmp, "-L", torch_lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda", "-L", BUILD, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding link failed (the C library is built):\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """The C library, for which nvcc is enough, and then the binding, for which there has to be a torch with CUDA: without
    one it is left out, and the calls that need it say so."""
    lib, binding = force or _lib_stale(), force or _binding_stale()
    if not (lib or binding):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ["-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"), "-lineinfo"]
    torch = _torch() if binding else None

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + common + ARCH + ["-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd = [cc, "-x", "c++"] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        compiled = ex.submit(_compile_binding, torch) if torch else None
        if lib:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".tmp{os.getpid()}"
            r = subprocess.run([cc, "-shared", "-cudart", "static"] + ARCH + objs + ["-o", tmp], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, LIB)
    if binding:
        if compiled:
            _link_binding(*compiled.result())
        elif verbose:
            sys.stderr.write("no torch with CUDA: the Python binding is left out\n")
        tmp = BINDING_STAMP + f".tmp{os.getpid()}"
        with open(tmp, "w") as f:
            f.write(f"{binding_key()}\n{'built' if compiled else 'left out'}\n")
        os.replace(tmp, BINDING_STAMP)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
