"""Build libswa.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m sliding_window_gqa_chunk_b200.csrc.build [--force] [--verbose]

The library links the CUDA runtime statically and reaches the driver API only
through cudaGetDriverEntryPoint, so it loads on a machine without a GPU.  Beside
it, _native.so is the Python module that takes torch tensors to the calls of the
8-bit cache and of the rotary positions (g++, against the installed torch).
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(HERE)
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libswa.so")
BINDING = os.path.join(PKG, "_native.so")

SOURCES = ["swa_api.cu", "swa_append.cu", "swa_decode.cu", "swa_prefill.cu", "swa_decode_static.cu",
           "swa_q8_api.cu", "swa_q8_cache.cu", "swa_q8_decode.cu", "swa_q8_decode_16.cu",
           "swa_q8_decode_64.cu", "swa_q8_decode_128.cu", "swa_rope.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(HERE, s) for s in SOURCES]
    files += glob.glob(os.path.join(HERE, "*.cuh")) + glob.glob(os.path.join(HERE, "*.h"))
    files += glob.glob(os.path.join(INCLUDE, "*.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build_binding(force: bool = False) -> str:
    """Build _native.so against the torch of this interpreter."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    src = os.path.join(HERE, "binding.cpp")
    inputs = [src, os.path.join(INCLUDE, "swa.h"), torch.__file__]
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in inputs):
        return BINDING
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    libs = cpp_extension.TORCH_LIB_PATH
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE]
    for path in [*cpp_extension.include_paths(), cuda, sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", path]
    cmd += [src, "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed building _native.so")
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, defines=(), out: str | None = None) -> str:
    """Build the library (into `out` when given, e.g. a checked-mode variant with
    extra preprocessor `defines` for the tests)."""
    target = out or LIB
    if out is None:
        build_binding(force)
    if not force and out is None and up_to_date():
        return LIB
    os.makedirs(os.path.dirname(os.path.abspath(target)), exist_ok=True)
    tmp = target + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC", "--threads", "0",
           "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
           "-I", INCLUDE, "-I", HERE, "-o", tmp]
    cmd += [f"-D{d}" for d in defines]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    cmd += [os.path.join(HERE, s) for s in SOURCES]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed building libswa.so")
    if verbose:
        sys.stderr.write(res.stderr)
    os.replace(tmp, target)
    return target


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
