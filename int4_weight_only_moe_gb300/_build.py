"""Build the CUDA library ``libmoe_w4a16.so`` in-tree for sm_103a with nvcc.

The translation units are compiled in parallel and linked into a shared
library next to this file (``int4_weight_only_moe_gb300/lib/``). That takes nvcc alone.
Beside it stands the extension module ``moe_w4a16_calls.so`` of the Python calls, where
torch is installed: the package works without it, small calls a few microseconds slower.
What is newer than its sources is not built again.
"""
from __future__ import annotations

import fcntl
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmoe_w4a16.so")
CALLS = os.path.join(LIBDIR, "moe_w4a16_calls.so")
SOURCES = ["pack.cu", "align.cu", "route.cu", "gemm.cu", "gemv.cu", "api.cu", "noalloc.cu",
           "route_scored.cu", "fp8_quant.cu", "fp8_matmul.cu", "fp8_many.cu", "ops_api.cu",
           "dispatch.cu", "route_backward.cu", "lora.cu", "lora_many.cu", "dispatch_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")
    return cand


def _inputs(*kinds):
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(kinds)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files + [os.path.abspath(__file__)]


def _newer(target, inputs) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB, _inputs(".cu", ".cuh"))


def _calls_up_to_date() -> bool:
    torch = _torch()
    if torch is None:
        return True
    try:
        with open(CALLS + ".txt") as f:
            return _newer(CALLS, _inputs(".cpp")) and f.read() == built_for(_version(torch))
    except OSError:
        return False


def up_to_date() -> bool:
    return _library_up_to_date() and _calls_up_to_date()


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if p.returncode != 0:
        raise RuntimeError("command failed:\n" + " ".join(cmd) + "\n" + p.stdout)
    return p.stdout


def _torch():
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec else None


def _version(torch: str) -> str:
    """torch.__version__, without the import."""
    spec = importlib.util.spec_from_file_location("torch_version", os.path.join(torch, "version.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return str(module.__version__)


def built_for(torch_version: str) -> str:
    """What the extension holds for: written beside it when it is built."""
    return f"torch {torch_version}, Python {sysconfig.get_config_var('EXT_SUFFIX')}\n"


def _build_calls(torch: str) -> None:
    """The extension module, against the library that stands there."""
    inc, obj, tmp = os.path.join(torch, "include"), os.path.join(BUILD, "calls.o"), CALLS + ".tmp"
    _run(["g++", "-std=c++17", "-O2", "-fPIC", "-w", "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-I", sysconfig.get_path("include"), "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj])
    _run(["g++", "-shared", "-o", tmp, obj, "-L", LIBDIR, "-lmoe_w4a16", "-L", os.path.join(torch, "lib"), "-ltorch_python",
          "-ltorch_cpu", "-ltorch", "-lc10", "-Wl,-rpath,$ORIGIN"])
    with open(CALLS + ".txt", "w") as f:
        f.write(built_for(_version(torch)))
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile what is needed; return the library's path. One process at a time: another one
    that builds here meanwhile waits, and finds it built."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    with open(os.path.join(BUILD, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)  # (given back when the file is closed)
        if force or not _library_up_to_date():
            _build_library(verbose, ptxas_info)
        if (torch := _torch()) and (force or not _calls_up_to_date()):
            try:
                _build_calls(torch)
            except (RuntimeError, OSError) as e:
                if os.path.exists(CALLS):
                    os.remove(CALLS)
                warnings.warn(f"the compiled Python calls could not be built, the Python steps are taken: {e}")
    return LIB


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        out = _run([cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj, out

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _, out in results:
            if out.strip():
                print(out)
    tmp = LIB + ".tmp"
    _run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"])
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
