"""Build libfa.so (sm_100a) in-tree with nvcc, and the serving operators' Python binding _serving.so with g++
against the torch that is installed (without one libfa.so is built alone).

Usage: python -m exact_io_aware_100_b200.build [--verbose]
"""
from __future__ import annotations

import importlib.metadata
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
EXT_FOR = os.path.join(PKG, "_serving.txt")     # the Python and torch it was built against
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


def torch_path() -> str | None:
    """Where a torch with CUDA is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    where = spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None
    return where if where and os.path.exists(os.path.join(where, "lib", "libc10_cuda.so")) else None


def extension_for(torch: str) -> str:
    """What _serving.so is compiled against, as one line: it loads with this Python and this torch only."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"{sysconfig.get_config_var('SOABI')}, torch {version} at {torch}"


def extension_command(torch: str) -> list[str]:
    include, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
            "-I", sysconfig.get_paths()["include"], "-I", include, "-I", os.path.join(include, "torch", "csrc", "api", "include"),
            "-I", cuda, "-o", EXT, EXT_SOURCE, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
            f"-Wl,-rpath,{lib}"]


def _newer(target: str, deps: list[str]) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def _header() -> str:
    return os.path.join(ROOT, "include", "fa.h")


def library_up_to_date() -> bool:
    return _newer(LIB, [os.path.join(CSRC, d) for d in DEPS] + [_header()])


def extension_up_to_date(torch: str) -> bool:
    if not _newer(EXT, [EXT_SOURCE, _header()]) or not os.path.exists(EXT_FOR):
        return False
    with open(EXT_FOR) as f:
        return f.read().strip() == extension_for(torch)


def up_to_date() -> bool:
    torch = torch_path()
    return library_up_to_date() and (torch is None or extension_up_to_date(torch))


def _run(what: str, cmd: list[str], verbose: bool) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"building {what} failed")


def build(force: bool = False, verbose: bool = False) -> str:
    """libfa.so first, which needs nvcc alone; then _serving.so, where there is a torch with CUDA to build it against."""
    if force or not library_up_to_date():
        _run("libfa.so", command(verbose), verbose)
    torch = torch_path()
    if torch is None:
        sys.stderr.write("no torch with CUDA: _serving.so, the Python binding of the serving operators, is not built\n")
    elif force or not extension_up_to_date(torch):
        _run("_serving.so", extension_command(torch), verbose)
        with open(EXT_FOR, "w") as f:
            f.write(extension_for(torch) + "\n")
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="--verbose" in sys.argv)
    print(LIB)
