"""The host code of the operators around the routed experts without a GPU: the compiled
objects linked to a fake CUDA runtime (fake_cuda_runtime.cpp) that logs what is launched."""
import ctypes
import os
import subprocess

import pytest

OBJECTS = ["route_scored.o", "fp8_quant.o", "fp8_matmul.o", "fp8_many.o", "ops_api.o"]
BUF = ctypes.c_void_p(4096)  # never read
F32, BF16 = 0, 1


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    from int4_weight_only_moe_gb300 import _build
    _build.build()
    objects = [os.path.join(_build.BUILD, o) for o in OBJECTS]
    if not all(map(os.path.exists, objects)):
        _build.build(force=True)
    out = str(tmp_path_factory.mktemp("fake") / "libops_fake.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-w", "-I", include, "-o", out,
                    os.path.join(here, "fake_cuda_runtime.cpp"), *objects, "-Wl,-Bsymbolic", "-Wl,-z,defs"], check=True)
    return out


@pytest.fixture
def lib(library, tmp_path):
    # (a copy of its own: nothing that the code keeps is left over from another test)
    path = str(tmp_path / "libops_fake.so")
    with open(library, "rb") as src, open(path, "wb") as dst:
        dst.write(src.read())
    L = ctypes.CDLL(path)
    from int4_weight_only_moe_gb300 import _SIGNATURES
    for name in ("moe_w4a16_fp8_matmul", "moe_w4a16_shared_expert", "moe_w4a16_fp8_status",
                 "moe_w4a16_fp8_plan_debug"):
        fn = getattr(L, name)
        fn.restype, fn.argtypes = _SIGNATURES[name]
    return L


def launched(lib):
    """(device, kernel, grid, cluster) of every launch so far."""
    out = []
    for i in range(lib.fake_launches()):
        dev, cluster, name, grid = ctypes.c_int(), ctypes.c_int(), ctypes.create_string_buffer(400), (ctypes.c_uint * 3)()
        lib.fake_launch(i, ctypes.byref(dev), name, 400, grid, ctypes.byref(cluster))
        out.append((dev.value, name.value.decode(), tuple(grid), cluster.value))
    return out


def matmul(lib, M, N, K, add=None, out=BUF, out_type=BF16):
    return lib.moe_w4a16_fp8_matmul(BUF, K, BUF, BUF, K, BUF, add, out, out_type, M, N, K, None)


def shared(lib, M, K, N):
    return lib.moe_w4a16_shared_expert(BUF, BUF, BUF, BUF, BUF, None, BUF, M, K, N, BUF, 1 << 40, None)


def test_every_device_is_set_up(lib):
    sizes = [(M, 4096, 7168) for M in (1, 20, 50, 100)] + [(4096, 4096, 1024), (4096, 4095, 1024)]
    seen = []
    for dev in (0, 1, 5, 0, 70):
        lib.fake_device(dev)
        lib.fake_clear()
        for M, N, K in sizes:
            assert matmul(lib, M, N, K) == 0, (dev, M)
            assert matmul(lib, M, N, K, add=BUF) == 0, (dev, M)
        for M in (1, 20, 50, 100, 4096):
            assert shared(lib, M, 1024, 512) == 0, (dev, M)
        got = launched(lib)
        assert {d for d, *_ in got} == {dev}
        seen.append([rest for _, *rest in got])
    assert all(s == seen[0] for s in seen)


def test_a_device_is_asked_once(lib):
    for dev in (0, 1):
        lib.fake_device(dev)
        matmul(lib, 1, 4096, 7168), matmul(lib, 4096, 4096, 1024)
        lib.fake_clear()
        matmul(lib, 1, 4096, 7168), matmul(lib, 4096, 4096, 1024)
        assert lib.fake_launches() == 2 and lib.fake_calls(b"cudaOccupancyMaxActiveClusters") == 0


KERNELS = {16: "few_kernelILi16E", 32: "few_kernelILi32E", 64: "few_kernelILi64E", 128: "few_kernelILi128E",
           256: "many_kernel", 0: "plain_kernel"}


@pytest.mark.parametrize("M", [1, 16, 17, 32, 40, 64, 65, 100, 200, 300, 700, 3000])
def test_the_plan_is_what_is_launched(lib, M):
    plan = (ctypes.c_int32 * 2)()
    for N, K in ((130, 16), (1024, 512), (4096, 7168), (2047, 272), (640, 1000)):
        for add in (None, BUF):
            for out in (BUF, ctypes.c_void_p(4098)):
                lib.fake_clear()
                assert matmul(lib, M, N, K, add=add, out=out) == 0
                assert lib.moe_w4a16_fp8_plan_debug(0, add, out, BF16, M, N, K, plan) == 0
                (_, kernel, _, cluster), = launched(lib)
                assert KERNELS[plan[0]] in kernel and plan[1] == cluster
    for K, N in ((256, 128), (7168, 2048), (2048, 384), (4096, 512)):
        lib.fake_clear()
        assert shared(lib, M, K, N) == 0
        _, up, down = launched(lib)
        assert lib.moe_w4a16_fp8_plan_debug(1, None, BUF, BF16, M, N, K, plan) == 0
        assert KERNELS[plan[0]] in up[1] and plan[1] == up[3]
        assert lib.moe_w4a16_fp8_plan_debug(2, None, BUF, BF16, M, K, N, plan) == 0
        assert KERNELS[plan[0]] in down[1] and plan[1] == down[3]


def test_plan_refusals(lib):
    plan = (ctypes.c_int32 * 2)()
    good = [0, None, BUF, BF16, 4, 128, 256, plan]
    for at, value, rc in [(0, 3, -1), (0, -1, -1), (3, 7, -1), (4, 0, -1), (5, 0, -1), (6, 0, -1), (5, 1 << 23, -2),
                          (7, None, -1)]:
        args = list(good)
        args[at] = value
        assert lib.moe_w4a16_fp8_plan_debug(*args) == rc
    assert lib.moe_w4a16_fp8_plan_debug(1, None, BUF, BF16, 4, 100, 256, plan) == -2


def test_status_clears_what_it_reports_and_nothing_else(lib):
    value = ctypes.c_int32(-1)
    lib.fake_status(0)
    assert lib.moe_w4a16_fp8_status(ctypes.byref(value), None) == 0 and value.value == 0
    # (clean: a product that gives up on another stream right now must still be seen)
    assert lib.fake_calls(b"cudaMemcpyAsync") == 1 and lib.fake_calls(b"cudaMemsetAsync") == 0
    lib.fake_status(2)
    assert lib.moe_w4a16_fp8_status(ctypes.byref(value), None) == 0 and value.value == 2
    assert lib.fake_calls(b"cudaMemsetAsync") == 1
    assert lib.moe_w4a16_fp8_status(ctypes.byref(value), None) == 0 and value.value == 0
