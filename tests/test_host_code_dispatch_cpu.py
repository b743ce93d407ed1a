"""The host code of the order, gather, combine, gradients and adapters without a GPU: the
compiled objects on the fake CUDA runtime (see test_host_code_cpu.py), which refuses a launch
with more shared memory than the kernel was allowed on its device."""
import ctypes
import os
import subprocess

import pytest

OBJECTS = ["route_scored.o", "fp8_quant.o", "fp8_matmul.o", "fp8_many.o", "ops_api.o", "dispatch.o", "route_backward.o", "lora.o",
           "lora_many.o", "dispatch_api.o"]
BUF, BUF2 = ctypes.c_void_p(4096), ctypes.c_void_p(1 << 45)  # of inputs and of outputs; never read
ODD, ODD2 = ctypes.c_void_p(4098), ctypes.c_void_p((1 << 45) + 2)
F32, BF16, E4M3 = 0, 1, 2
DEVICES = (0, 1, 5, 0, 70)
NAMES = [n for n in ("moe_w4a16_dispatch_sort", "moe_w4a16_dispatch_gather", "moe_w4a16_dispatch_sort_gather",
                     "moe_w4a16_combine", "moe_w4a16_combine_backward", "moe_w4a16_route_scored_backward", "moe_w4a16_lora",
                     "moe_w4a16_lora_workspace_size")]


@pytest.fixture(scope="module")
def library(tmp_path_factory):
    from int4_weight_only_moe_gb300 import _build
    _build.build()
    objects = [os.path.join(_build.BUILD, o) for o in OBJECTS]
    if not all(map(os.path.exists, objects)):
        _build.build(force=True)
    out = str(tmp_path_factory.mktemp("fake") / "libdispatch_fake.so")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-w", "-I", include, "-o", out,
                    os.path.join(here, "fake_cuda_runtime.cpp"), *objects, "-Wl,-Bsymbolic", "-Wl,-z,defs"], check=True)
    return out


@pytest.fixture
def lib(library, tmp_path):
    path = str(tmp_path / "libdispatch_fake.so")
    with open(library, "rb") as src, open(path, "wb") as dst:
        dst.write(src.read())
    L = ctypes.CDLL(path)
    from int4_weight_only_moe_gb300 import _SIGNATURES
    for name in NAMES:
        fn = getattr(L, name)
        fn.restype, fn.argtypes = _SIGNATURES[name]
    return L


def launched(lib):
    out = []
    for i in range(lib.fake_launches()):
        dev, cluster, name, grid = ctypes.c_int(), ctypes.c_int(), ctypes.create_string_buffer(400), (ctypes.c_uint * 3)()
        lib.fake_launch(i, ctypes.byref(dev), name, 400, grid, ctypes.byref(cluster))
        out.append((dev.value, name.value.decode(), tuple(grid), cluster.value))
    return out


def lora(lib, M, K=512, N=512, r=16, L=4, add=BUF, add_type=BF16, out=BUF2, out_type=BF16, x=BUF, ws=BUF):
    return lib.moe_w4a16_lora(x, K, BUF, BUF, BUF, BUF, add, add_type, out, out_type, M, K, N, r, L, ws, 1 << 40, None)


def sort(lib, M, topk, E, block=1):
    return lib.moe_w4a16_dispatch_sort(BUF, M, topk, 0, E, block, BUF2, BUF2, BUF2, None)


def sort_gather(lib, M, topk, E, block=1, K=512, kind=BF16, x=BUF):
    return lib.moe_w4a16_dispatch_sort_gather(x, kind, K, BUF, M, K, topk, 0, E, block, BUF2, BUF2, BUF2, BUF2, None)


def test_every_device_is_set_up(lib):
    seen = []
    for dev in DEVICES:
        lib.fake_device(dev)
        lib.fake_clear()
        for M in (1, 100, 300, 1000, 5000, 20000):
            for E in (1, 384, 1024):
                assert sort(lib, M, 8, E) == 0 and sort_gather(lib, M, 8, E, 16) == 0
            for r in (1, 8, 16, 24, 32, 48, 64, 72, 96, 128):
                for add, out in ((BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32), (None, F32), (None, BF16)):
                    assert lora(lib, M, r=r, add=None if add is None else BUF, add_type=add or 0, out_type=out) == 0, (dev, M, r)
        got = launched(lib)
        assert {d for d, *_ in got} == {dev}
        seen.append([rest for _, *rest in got])
    assert all(s == seen[0] for s in seen)


def kernels(lib, call):
    lib.fake_clear()
    assert call() == 0
    return [(name, grid, cluster) for _, name, grid, cluster in launched(lib)]


def test_adapters_take_the_kernel_of_their_size(lib):
    for M, r, name in ((1, 16, "few"), (768, 64, "few"), (384, 128, "few"), (40, 8, "few")):
        (k, grid, cluster), = kernels(lib, lambda: lora(lib, M, r=r))
        assert "lora_few" in k and cluster == 8 and grid[0] % 8 == 0
    for M, r in ((769, 64), (385, 128), (1536, 16)):
        (k, grid, cluster), = kernels(lib, lambda: lora(lib, M, r=r))
        assert "lora_many" in k and grid[0] % cluster == 0 and grid[0] // cluster >= (M + 127) // 128
    for M, r in ((1537, 64), (8192, 16), (100000, 64)):
        (s, _, _), (k, grid, cluster) = kernels(lib, lambda: lora(lib, M, r=r))
        assert "sort" in s and "lora_many" in k and grid[0] % cluster == 0
        assert grid[0] // cluster >= (M + 127) // 128
    # what cannot be read in pieces goes value by value, as many rows at a time as few are
    for kw, whole in ((dict(K=513), 0), (dict(N=514), 0), (dict(r=3), 0), (dict(r=12), 1), (dict(x=ODD), 0), (dict(out=ODD2), 0),
                      (dict(add=ODD), 0), (dict(r=100, N=514), 0)):
        for M in (5, 768, 5000):
            got = kernels(lib, lambda: lora(lib, M, **kw))
            assert len(got) == -(-M // (384 if kw.get("r") == 100 else 768))
            assert all("lora_few" in k and f"Lb{whole}E" in k and grid[0] % 8 == 0 for k, grid, _ in got)
    assert lib.moe_w4a16_lora_workspace_size(1536, 512, 512, 64, 4) == 0
    assert lib.moe_w4a16_lora_workspace_size(1537, 512, 512, 64, 4) > 0


def test_rows_of_an_adapter_alone_in_its_group_have_a_cluster(lib):
    for M, L in ((1, 1023), (30, 8), (64, 32), (700, 1023), (700, 3), (33, 2)):
        (_, grid, _), = kernels(lib, lambda: lora(lib, M, L=L))
        groups = min(M, L + 1 + -(-M // 16))
        assert grid[0] == 8 * groups


def test_few_slots_take_one_launch(lib):
    for M, topk, n in ((1, 8, 1), (128, 8, 1), (129, 8, 2), (32, 32, 1), (33, 32, 2), (8192, 8, 2)):
        for block in (1, 128):
            assert len(kernels(lib, lambda: sort_gather(lib, M, topk, 384, block))) == n


def test_pieces_go_by_alignment(lib):
    for K, kind, x, piece in ((512, BF16, BUF, 16), (514, BF16, BUF, 4), (513, BF16, BUF, 2), (513, E4M3, BUF, 1), (512, BF16, ODD, 2),
                              (513, F32, BUF, 4)):
        for M in (4, 4000):
            got = kernels(lib, lambda: sort_gather(lib, M, 8, 64, K=K, kind=kind, x=x))
            assert f"ILi{piece}E" in got[-1][0], (K, kind, M)


def test_combine_and_gradients_launch_once(lib):
    for M in (1, 90, 9000):
        for y, out in ((BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)):
            for K, wide in ((512, "Li8E"), (516, "Li1E")):
                (k, grid, _), = kernels(lib, lambda: lib.moe_w4a16_combine(BUF, y, BUF, BUF, BUF, BUF2, out, M, K, 8, 99, None))
                assert wide in k and grid[0] % M == 0
                (k, grid, _), = kernels(lib, lambda: lib.moe_w4a16_combine_backward(BUF, out, BUF, y, BUF, BUF, BUF, BUF, BUF2, BUF2, M, K, 8,
                                                                                     64, 128, None))
                assert wide in k and grid[0] == M + 64 * 8
        for topk, scoring, renorm, name in ((8, 1, 1, "Li8E"), (9, 1, 1, "Li16E"), (32, 0, 1, "Li32E"), (8, 0, 0, "plain"), (8, 1, 0, "Li8E")):
            (k, _, _), = kernels(lib, lambda: lib.moe_w4a16_route_scored_backward(BUF, BUF, F32, 64, BUF, M, 64, topk, scoring, renorm, 1.0,
                                                                                  BUF2, None))
            assert name in k
