"""Build libfa.so (sm_100a) in-tree with nvcc, and the serving operators' binding _serving.so with g++.

Usage: python -m exact_io_aware_100_b200.build [--verbose]
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libfa.so")
EXT = os.path.join(PKG, "_serving.so")          # the binding of the serving operators, against torch's headers
EXT_SOURCE = os.path.join(CSRC, "serving_binding.cpp")
SOURCES = ["fa_lib.cu"]
DEPS = ["fa_lib.cu", "fa_api.cu", "serving_api.cuh", "rotary_kernel.cuh", "paged_decode_kernel.cuh", "pages_kernel.cuh",
        "fwd_kernel.cuh", "bwd_kernel.cuh", "bwd256_kernel.cuh", "decode_kernel.cuh", "decode_warp_kernel.cuh", "fwd64_kernel.cuh", "fwd256_kernel.cuh", "layout.cuh",
        "ptx.cuh"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def command(verbose: bool = False) -> list[str]:
    cmd = [nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
           "-std=c++17", "-shared", "-Xcompiler", "-fPIC,-O2", "-cudart", "static",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-o", LIB] + [os.path.join(CSRC, s) for s in SOURCES]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    return cmd


def extension_command() -> list[str]:
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    include, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
            "-I", sysconfig.get_paths()["include"], "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
            "-I", cuda, "-o", EXT, EXT_SOURCE, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            f"-Wl,-rpath,{lib}"]


def _newer(target: str, deps: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    header = os.path.join(ROOT, "include", "fa.h")
    return _newer(LIB, [os.path.join(CSRC, d) for d in DEPS] + [header]) and _newer(EXT, [EXT_SOURCE, header])


def build(force: bool = False, verbose: bool = False) -> str:
    header = os.path.join(ROOT, "include", "fa.h")
    for what, cmd, target, deps in (
            ("libfa.so", command(verbose), LIB, [os.path.join(CSRC, d) for d in DEPS] + [header]),
            ("_serving.so", extension_command(), EXT, [EXT_SOURCE, header])):
        if not force and _newer(target, deps):
            continue
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"building {what} failed")
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
