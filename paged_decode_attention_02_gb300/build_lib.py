"""Builds ``libpda.so`` in-tree from ``csrc/*.cu`` with nvcc for sm_103a.

Each translation unit is compiled in parallel to ``_build/`` and linked with
``nvcc -shared`` (static CUDA runtime, so the library needs no LD_LIBRARY_PATH). Beside it the
host compiler builds ``_marshal``, the extension module that hands tensors to the library's short
calls; its file name says for which torch and Python, so that another of them asks for a file of
its own. Run as
``python -m paged_decode_attention_02_gb300.build_lib`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libpda.so")
MARSHAL_SRC = os.path.join(PKG, "marshal", "marshal.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _defines():
    """Extra -D options from PDA_NVCC_DEFINES (space-separated NAME=VALUE), for tuning builds
    (the csrc macros PDA_ATTN_WARPS, PDA_TC_PAIR_WARPS_*, PDA_PACK_TOKENS, ...)."""
    return ["-D" + d for d in os.environ.get("PDA_NVCC_DEFINES", "").split() if d]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "pda.h"), __file__]


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path)
                                        for d in deps)


def up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def marshal_path() -> str:
    """The extension module of the torch and Python that run now."""
    import torch

    abi = "" if torch._C._GLIBCXX_USE_CXX11_ABI else "-oldabi"
    return os.path.join(PKG, f"_marshal-torch{torch.__version__}{abi}" +
                        (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def marshal_up_to_date() -> bool:
    return _newer(marshal_path(), [MARSHAL_SRC, os.path.join(INCLUDE, "pda.h"), __file__])


def _build_marshal():
    """The extension module: torch's and Python's headers, no CUDA code."""
    import torch

    path = marshal_path()
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no host C++ compiler")
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    lib = os.path.join(root, "lib")
    tmp = path + f".tmp{os.getpid()}"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + INCLUDE, "-isystem", cuda,
           "-isystem", os.path.join(root, "include"), "-isystem",
           os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", MARSHAL_SRC, "-o",
           tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + lib]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {path} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not up to date and returns the library's path. Where only the extension module
    cannot be built, the library is in place when this raises, and the calls through it work."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        marshal = None if not force and marshal_up_to_date() else ex.submit(_build_marshal)
        if force or not up_to_date():
            _build_library(verbose)
        if marshal is not None:
            marshal.result()
    return LIB_PATH


def _build_library(verbose: bool):
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *_defines(), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
