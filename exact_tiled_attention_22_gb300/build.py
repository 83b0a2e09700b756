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
STAMP = os.path.join(BUILD, "attn_bind.stamp")
SOURCES = ["attn_api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_decode.cu", "attn_noalloc.cu", "attn_diag.cu",
           "attn_pages.cu", "attn_kv8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         f"-I{os.path.join(ROOT, 'include')}"] + ARCH


def _nvcc_path() -> str:
    return shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


def nvcc() -> str:
    exe = _nvcc_path()
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn.so")
    return exe


def _newer(lib, files) -> bool:
    return os.path.exists(lib) and all(os.path.getmtime(f) <= os.path.getmtime(lib) for f in files)


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def lib_up_to_date() -> bool:
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return _newer(LIB, files + _headers())


def _stamp() -> str:
    """What attn_bind.so was built for besides its sources: this torch (its version.py
    names version, commit and CUDA), this Python and this toolkit."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return "\n".join([sysconfig.get_config_var("SOABI") or "", _torch_dir(), _nvcc_path(), f.read()])


def bind_up_to_date() -> bool:
    if not _newer(BIND, [BIND_SRC] + _headers()) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == _stamp()


def up_to_date() -> bool:
    return lib_up_to_date() and bind_up_to_date()


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
    with open(STAMP, "w") as f:
        f.write(_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not up to date.  libattn.so is in place before an error in
    attn_bind.so's build (a torch without its C++ headers, say) is raised."""
    todo_lib, todo_bind = force or not lib_up_to_date(), force or not bind_up_to_date()
    if not todo_lib and not todo_bind:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    bind_obj = os.path.join(BUILD, "attn_bind.o")

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        r = _run([nvcc()] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj], f"nvcc failed on {src}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bind = ex.submit(compile_bind, bind_obj) if todo_bind else None
        if todo_lib:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([nvcc(), "-shared"] + ARCH + ["-o", tmp] + objs, "link failed")
            os.replace(tmp, LIB)
        if bind is not None:
            bind.result()
            link_bind(bind_obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
