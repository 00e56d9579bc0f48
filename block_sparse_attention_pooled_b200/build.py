"""Builds libsparge.so in-tree with nvcc for sm_100a (one translation unit), and the compiled binding of its newer
entry points, _bind, against it and torch."""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "sparge.cu")
HEADERS = [os.path.join(PKG, "csrc", f) for f in ("ptx.cuh", "mask.cuh", "attn.cuh", "linear.cuh", "lin_out.cuh", "lin_bwd.cuh", "quant.cuh", "attn_q8.cuh", "attn_bwd.cuh", "selftest.cuh", "window.cuh", "cache.cuh", "cache_sched.cuh", "cache_attn.cuh", "cache_chunk.cuh", "wattn.cuh", "wattn_bwd.cuh", "window_host.cuh")] + [
    os.path.join(ROOT, "include", "sparge.h")
]
LIB = os.path.join(PKG, "libsparge.so")
BIND_SRC = os.path.join(PKG, "csrc", "bind.cpp")
BIND = os.path.join(PKG, "_bind" + sysconfig.get_config_var("EXT_SUFFIX"))
BIND_FOR = os.path.join(PKG, "_build", "bind_for.txt")  # the torch and Python that _bind was built for

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.exists(f) and os.path.getmtime(f) > t for f in [SRC, *HEADERS])


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _stale():
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"), SRC, "-o", tmp]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.check_call(cmd, stdout=None if verbose else subprocess.DEVNULL)
        os.replace(tmp, LIB)
    if force or _bind_stale():
        _build_bind()
        os.makedirs(os.path.dirname(BIND_FOR), exist_ok=True)
        with open(BIND_FOR, "w") as f:
            f.write(_bind_target())
    return LIB


def _bind_target() -> str:
    """What the binding has to be built for; its name holds no more than the Python version."""
    return f"torch {importlib.metadata.version('torch')}, Python {sys.version.split()[0]}"


def _bind_stale() -> bool:
    if not (os.path.exists(BIND) and os.path.exists(BIND_FOR)):
        return True
    with open(BIND_FOR) as f:
        if f.read() != _bind_target():
            return True
    deps = [BIND_SRC, os.path.join(ROOT, "include", "sparge.h")]
    return any(os.path.getmtime(f) > os.path.getmtime(BIND) for f in deps)


def _build_bind() -> None:
    import torch

    base = os.path.dirname(torch.__file__)
    lib = os.path.join(base, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    tmp = BIND + f".tmp{os.getpid()}"
    subprocess.check_call([
        shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_bind",
        "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
        "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, BIND_SRC, "-o", tmp,
        "-L", PKG, "-l:libsparge.so", "-Wl,-rpath,$ORIGIN",
        "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
    ])
    os.replace(tmp, BIND)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
