"""Builds libattn.so in-tree from csrc/ with nvcc for sm_103a only, and the
Python module attn_bind.so (csrc/attn_bind.cpp, host code on torch's C++ headers).

Each translation unit is compiled in parallel into _build/, then linked into
exact_tiled_attention_22_gb300/libattn.so.  A rebuild happens only when a
source or header is newer than the libraries.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libattn.so")
BIND = os.path.join(HERE, "attn_bind.so")
BIND_SRC = os.path.join(CSRC, "attn_bind.cpp")
SOURCES = ["attn_api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_decode.cu", "attn_noalloc.cu", "attn_diag.cu",
           "attn_pages.cu", "attn_kv8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{os.path.join(ROOT, 'include')}"] + ARCH


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn.so")
    return exe


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files += glob.glob(os.path.join(ROOT, "include", "*.h"))
    files += [os.path.abspath(__file__), BIND_SRC]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BIND):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: attn_bind.so is built on its headers")
    return list(spec.submodule_search_locations)[0]


def compile_bind(obj: str) -> None:
    inc = os.path.join(_torch_dir(), "include")
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-c", BIND_SRC, "-o", obj,
          f"-I{os.path.join(ROOT, 'include')}", f"-I{sysconfig.get_paths()['include']}", f"-I{inc}",
          f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
          f"-I{os.path.join(os.path.dirname(os.path.dirname(nvcc())), 'include')}"], f"g++ failed on {BIND_SRC}")


def link_bind(obj: str) -> None:
    """Against libattn.so beside it: the one that the ctypes binding loads."""
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BIND + f".tmp{os.getpid()}"
    _run([shutil.which("g++") or "g++", "-shared", obj, "-o", tmp, f"-L{HERE}", "-l:libattn.so", "-Wl,-rpath,$ORIGIN",
          f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "link of attn_bind.so failed")
    os.replace(tmp, BIND)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    exe = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [exe] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    bind_obj = os.path.join(BUILD, "attn_bind.o")
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(compile_bind, bind_obj)
        objs = list(ex.map(compile_one, SOURCES))
        bind.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [exe, "-shared"] + ARCH + ["-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    link_bind(bind_obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
