"""Build the CUDA library ``libmoe_w4a16.so`` in-tree for sm_103a with nvcc.

The translation units are compiled in parallel and linked into a shared
library next to this file (``int4_weight_only_moe_gb300/lib/``), and beside it the
extension module ``moe_w4a16_calls.so`` of the Python calls. A rebuild is
skipped when both are newer than every source and header.
"""
from __future__ import annotations

import os
import importlib.util
import shutil
import subprocess
import sysconfig
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


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".cpp"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return files + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if p.returncode != 0:
        raise RuntimeError("command failed:\n" + " ".join(cmd) + "\n" + p.stdout)
    return p.stdout


def _torch() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is needed to build the Python calls")
    return list(spec.submodule_search_locations)[0]


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile the library if needed; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        out = _run([cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj])
        return obj, out

    calls = os.path.join(BUILD, "calls.o")

    def compile_calls():
        inc = os.path.join(_torch(), "include")
        _run(["g++", "-std=c++17", "-O2", "-fPIC", "-w", "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
              "-I", sysconfig.get_path("include"), "-c", os.path.join(CSRC, "calls.cpp"), "-o", calls])

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        module = ex.submit(compile_calls)
        results = list(ex.map(compile_one, SOURCES))
        module.result()
    if verbose or ptxas_info:
        for _, out in results:
            if out.strip():
                print(out)
    tmp = LIB + ".tmp"
    _run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"])
    os.replace(tmp, LIB)
    tmp = CALLS + ".tmp"
    _run(["g++", "-shared", "-o", tmp, calls, "-L", LIBDIR, "-lmoe_w4a16", "-L", os.path.join(_torch(), "lib"), "-ltorch_python",
          "-ltorch_cpu", "-ltorch", "-lc10", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, CALLS)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
