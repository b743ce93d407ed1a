"""Tensors of torch's function transforms in the compiled Python calls, without a GPU. Such a
tensor has the plain type, a shape and strides, but no storage: asking for its address raises,
or gives 0, which the C entries take for an optional tensor that is not given. The calls have to hand it back like anything else that is not plainly right. The source is
compiled here without its device test, on C entries that only count their calls, and run in
another process: a call that throws without the interpreter's lock ends it."""
import os
import subprocess
import sys
import sysconfig

import pytest
import torch

NAMES = ["gather", "sort_gather", "combine", "combine_backward", "route_backward", "lora"]

ENTRIES = """
#include "moe_w4a16.h"
extern "C" {
long long moe_w4a16_dispatch_rows(int M, int topk, int E, int block) {
  const long long n = static_cast<long long>(M) * topk;
  return n + (n < E ? n : E) * (block - 1LL);
}
size_t moe_w4a16_lora_workspace_size(int, int, int, int, int) { return 0; }
int moe_w4a16_dispatch_gather(const void*, int, long long, const int32_t*, const int32_t*, const int32_t*, void*, int, int, int, int,
                              int, void*) { return 0; }
int moe_w4a16_dispatch_sort_gather(const void*, int, long long, const int32_t*, int, int, int, int, int, int, int32_t*, int32_t*,
                                   int32_t*, void*, void*) { return 0; }
int moe_w4a16_combine(const void*, int, const float*, const int32_t*, const void*, void*, int, int, int, int, int, void*) { return 0; }
int moe_w4a16_combine_backward(const void*, int, const void*, int, const float*, const int32_t*, const int32_t*, const int32_t*,
                               void*, float*, int, int, int, int, int, void*) { return 0; }
int moe_w4a16_route_scored_backward(const float*, const void*, int, long long, const int32_t*, int, int, int, int, int, float, void*,
                                    void*) { return 0; }
int moe_w4a16_lora(const uint16_t*, long long, const uint16_t*, const uint16_t*, const float*, const int32_t*, const void*, int,
                   void*, int, int, int, int, int, int, void*, size_t, void*) { return 0; }
}
"""

SCRIPT = """
import importlib.machinery, importlib.util, sys
import torch
name, path = sys.argv[1:]
loader = importlib.machinery.ExtensionFileLoader("moe_w4a16_calls", path)
calls = importlib.util.module_from_spec(importlib.util.spec_from_file_location("moe_w4a16_calls", path, loader=loader))
loader.exec_module(calls)
B, F, I = torch.bfloat16, torch.float32, torch.int32
M, K, E, TOPK, BLOCK = 4, 32, 5, 2, 3
R = M * TOPK + E * (BLOCK - 1)
t = lambda dtype, *shape: torch.zeros(*shape, dtype=dtype)
order = [t(I, E + 1), t(I, R), t(I, M, TOPK)]
args = dict(
    gather=[t(B, M, K), *order, t(B, R, K)],
    sort_gather=[t(B, M, K), t(I, M, TOPK), E, 0, BLOCK, *order, t(B, R, K)],
    combine=[t(B, R, K), t(F, M, TOPK), order[1], order[2], t(F, M, K), t(F, M, K)],
    combine_backward=[t(F, M, K), t(B, R, K), t(F, M, TOPK), *order, t(B, R, K), t(F, M, TOPK)],
    route_backward=[t(F, M, TOPK), t(F, M, E), t(I, M, TOPK), 1, True, 2.5, t(F, M, E)],
    lora=[t(B, M, K), t(B, 3, 8, K), t(B, 3, 16, 8), t(I, M), t(F, M, 16), t(F, 3), t(B, M, 16), 1 << 20])[name]
call = lambda args: getattr(calls, name)(-1, 0, *args)  # (-1: where a tensor of the host says it is)
assert call(args) == 0
APPLY = dict(vmap=lambda f, x: torch.vmap(f)(torch.stack([x, x])), grad=lambda f, x: torch.func.grad(f)(x),
             vjp=lambda f, x: torch.func.vjp(f, x), jvp=lambda f, x: torch.func.jvp(f, (x,), (x,)),
             functionalize=lambda f, x: torch.func.functionalize(f)(x))
for how, apply in APPLY.items():
    tried = 0
    for at, arg in enumerate(args):
        if not torch.is_tensor(arg) or not (arg.is_floating_point() or how in ("vmap", "functionalize")):
            continue
        print(how, at, file=sys.stderr, flush=True)
        def one(x):
            got = call([*args[:at], x, *args[at + 1:]])
            assert got is None, got
            return x.sum()
        apply(one, arg)
        tried += 1
    assert tried >= 2
def every(*ts):
    left = list(ts)
    assert call([left.pop(0) if torch.is_tensor(a) else a for a in args]) is None
    return ts[0].sum()
torch.vmap(every)(*[torch.stack([a, a]) for a in args if torch.is_tensor(a)])
assert call(args) == 0
"""


@pytest.fixture(scope="module")
def module(tmp_path_factory):
    from int4_weight_only_moe_gb300 import _build
    with open(os.path.join(_build.CSRC, "calls.cpp")) as f:
        source = f.read()
    assert source.count("!t.is_cuda()") == 1
    source = source.replace("!t.is_cuda()", "false").replace('"../../include/moe_w4a16.h"', '"moe_w4a16.h"')
    where = tmp_path_factory.mktemp("calls")
    (where / "calls.cpp").write_text(source)
    (where / "entries.cpp").write_text(ENTRIES)
    root = os.path.dirname(torch.__file__)
    out = str(where / "calls.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-w", "-I", _build.INCLUDE, "-I", os.path.join(root, "include"),
                    "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", sysconfig.get_path("include"),
                    "-o", out, str(where / "calls.cpp"), str(where / "entries.cpp"), "-L", os.path.join(root, "lib"),
                    "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"], check=True)
    (where / "run.py").write_text(SCRIPT)
    return str(where / "run.py"), out


@pytest.mark.parametrize("name", NAMES)
def test_tensors_without_storage_are_handed_back(module, name):
    run, out = module
    got = subprocess.run([sys.executable, run, name, out], capture_output=True, text=True)
    assert got.returncode == 0, (got.returncode, got.stderr[-2000:])
