"""Build libflce.so in-tree with nvcc for sm_103a, and beside it the PyTorch
operators of its differentiable layer norm and scores (host code, g++).

    python -m chunked_lm_head_gb300.build          # build if sources changed
    python -m chunked_lm_head_gb300.build --force  # rebuild

Both are written to chunked_lm_head_gb300/_build/ (git-ignored).
"""
from __future__ import annotations

import argparse
import importlib.metadata
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libflce.so")


def _torch_version() -> str | None:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None  # the C library alone


# (its name carries the PyTorch it was compiled against)
TORCH_LIB_PATH = os.path.join(BUILD_DIR, f"flce_torch-{_torch_version()}.so")
TORCH_SOURCE = os.path.join(CSRC, "torch_ops.cpp")
SOURCES = ["flce.cu"]
HEADERS = ["ptx.cuh", "gemm.cuh", "small_kernels.cuh", "host_common.cuh", "options.cuh", "plan.cuh",
           "launch.cuh", "norm.cuh", "norm_api.cuh", "layer_norm.cuh", "layer_norm_api.cuh", "topk.cuh", "topk_api.cuh",
           "score.cuh", "score_api.cuh"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libflce")


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "flce.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer(target: str, inputs: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB_PATH, _inputs())


def torch_ops_up_to_date() -> bool:
    return _newer(TORCH_LIB_PATH, [TORCH_SOURCE, os.path.join(INCLUDE, "flce.h"), os.path.abspath(__file__)])


def _start_torch_ops(tmp: str) -> subprocess.Popen:
    import torch
    from torch.utils import cpp_extension
    flags = [f for d in cpp_extension.include_paths() for f in ("-isystem", d)]
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")  # the stream's type
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE, *flags, "-isystem", cuda,
           "-o", tmp, TORCH_SOURCE, f"-L{libs}", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build_torch_ops(force: bool = False) -> str:
    """Compile the PyTorch operators alone (skipped when up to date); returns their path."""
    if not force and torch_ops_up_to_date():
        return TORCH_LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = TORCH_LIB_PATH + f".tmp{os.getpid()}"
    _finish_torch_ops(_start_torch_ops(tmp), tmp)
    return TORCH_LIB_PATH


def _finish_torch_ops(proc: subprocess.Popen, tmp: str) -> None:
    out, _ = proc.communicate()
    if proc.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(proc.args) + "\n" + out)
    os.replace(tmp, TORCH_LIB_PATH)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libflce.so and the PyTorch operators, at the same time (each skipped
    when up to date); returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    ops = None
    if _torch_version() is not None and (force or not torch_ops_up_to_date()):
        ops_tmp = TORCH_LIB_PATH + f".tmp{os.getpid()}"
        ops = _start_torch_ops(ops_tmp)
    try:
        return _build_library(force, verbose)
    finally:
        if ops is not None:
            _finish_torch_ops(ops, ops_tmp)


def _build_library(force: bool, verbose: bool) -> str:
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc_path(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--shared",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "-Xptxas", "-v" if verbose else "-O3",
           "-I", INCLUDE, "-I", CSRC, "-DFLCE_BUILDING_LIBRARY",
           "-o", tmp] + [os.path.join(CSRC, s) for s in SOURCES]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))
