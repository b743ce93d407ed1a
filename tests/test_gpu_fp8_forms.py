"""The forms of the 8-bit products at sizes that reach each of them, against the float64
definitions. Tolerances as in test_gpu_fp8.py."""
import pytest
import torch

import int4_weight_only_moe_gb300 as pkg
from int4_weight_only_moe_gb300 import BF16, F32, fp8, routing
from tests.gpu_helpers import assert_close, bf16_tensor_to_f64
from tests.test_gpu_fp8 import (_built, check_product, expert, expert_reference, operands,  # noqa: F401 (a fixture)
                                rand)

pytestmark = pytest.mark.gpu


def test_launches_back_to_back_keep_their_results():
    # (a product's CTAs hand their shared memory to the next launch's while others still run:
    # pairs of CTAs, clusters and single ones in turn, each right every time)
    shapes = [(2048, 1024, 384), (4, 512, 2048), (1500, 2048, 128), (40, 640, 1024), (100, 256, 1024), (700, 4096, 256)]
    ops = [operands(*shape, seed=i) for i, shape in enumerate(shapes)]
    first = [fp8.matmul(*o) for o in ops]
    for out, o in zip(first, ops):
        check_product(out, *o)
    for _ in range(40):
        outs = [fp8.matmul(*o) for o in ops]
        assert all(torch.equal(a, b) for a, b in zip(outs, first))
    assert fp8.status() == 0


def plan(stage, M, N, K, out_type=BF16, add=None, out=None):
    """Rows of a tile of the kernel that a product takes (256: the many-row kernel)."""
    return pkg.moe_w4a16_fp8_plan_debug(stage, add, out, out_type, M, N, K)[0]


def shifted(shape, by, dtype=torch.bfloat16):
    """A zeroed tensor that begins `by` elements into an allocation, and the allocation."""
    n = shape[0] * shape[1]
    buf = torch.zeros(n + 64, dtype=dtype, device="cuda")
    return buf[by:by + n].view(shape), buf


# M, N, K, out type, addend, elements by which the output (and addend) begin into an allocation:
# whole pieces and any alignment, with and without addends; one tile to a pair of CTAs, then two
# to four (76 pairs), several blocks of the reduction to each
MANY = [(2048, 2048, 128, BF16, True, 0), (3001, 2047, 272, BF16, False, 0), (3001, 2047, 272, BF16, True, 0),
        (3001, 2047, 272, BF16, True, 1), (4097, 1003, 400, F32, True, 0), (2049, 2047, 144, BF16, False, 0),
        (2049, 1024, 272, F32, False, 0), (2500, 2048, 272, BF16, True, 1), (2500, 2048, 272, F32, False, 1),
        (3841, 4096, 384, BF16, False, 0), (3841, 4096, 384, BF16, True, 0), (3700, 4095, 400, BF16, True, 0),
        (3700, 4033, 272, F32, False, 3), (3700, 3999, 272, F32, True, 1)]


@pytest.mark.parametrize("M,N,K,kind,with_add,off", MANY)
def test_product_of_many_rows(M, N, K, kind, with_add, off):
    dtype = torch.bfloat16 if kind == BF16 else torch.float32
    ops = operands(M, N, K, M + N)
    out, buf = shifted((M, N), off, dtype)
    add = shifted((M, N), off)[0].copy_(rand((M, N), 5)) if with_add else None
    assert plan(0, M, N, K, kind, add, out) == 256
    fp8.matmul(*ops, add=add, out=out)
    check_product(out, *ops, add=add)
    assert not buf[:off].any() and not buf[off + M * N:].any()
    if with_add and kind == BF16:  # in place
        mine, buf = shifted((M, N), off)
        mine.copy_(add)
        fp8.matmul(*ops, add=mine, out=mine)
        assert torch.equal(mine, out)
        assert not buf[:off].any() and not buf[off + M * N:].any()


# tokens, hidden size, features, rows of a tile of the gate/up product
EXPERTS = [(9, 512, 256, 16), (30, 512, 256, 32), (60, 512, 256, 64), (70, 7168, 256, 128), (100, 1536, 128, 128),
           (200, 2048, 384, 128), (700, 4096, 512, 128), (3700, 384, 2048, 256), (5000, 256, 1536, 256)]


@pytest.mark.parametrize("M,K,N,rows", EXPERTS)
def test_shared_expert_of_each_form(M, K, N, rows):
    assert plan(1, M, N, K) == rows
    w, x, add = expert(K, N, M), rand((M, K), 2), rand((M, K), 3)
    out = fp8.shared_expert(x, *w, add=add)
    assert_close(bf16_tensor_to_f64(out), expert_reference(x, w, add), "shared expert + routed")
    fp8.shared_expert(x, *w, add=add, out=add)
    assert torch.equal(add, out)


def gives_up(call):
    want = call().clone()
    assert fp8.status() == 0
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 1000)
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_TEST_WAIT_NEVER_COMPLETES, 1)
    try:
        call()
        assert fp8.status() == pkg.STATUS_TIMEOUT
    finally:
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_TEST_WAIT_NEVER_COMPLETES, 0)
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 0)
    assert torch.equal(call(), want) and fp8.status() == 0


@pytest.mark.parametrize("M,N,K,kind,with_add", [c[:5] for c in MANY[:3]] + [(3001, 2047, 272, F32, False)])
def test_wait_limit_of_products_of_many_rows(M, N, K, kind, with_add):
    ops, add = operands(M, N, K, 1), rand((M, N), 2) if with_add else None
    dtype = torch.bfloat16 if kind == BF16 else torch.float32
    assert plan(0, M, N, K, kind, add) == 256
    gives_up(lambda: fp8.matmul(*ops, add=add, out_dtype=dtype))


@pytest.mark.parametrize("M,K,N,rows", EXPERTS)
def test_wait_limit_of_shared_experts(M, K, N, rows):
    assert plan(1, M, N, K) == rows
    w, x = expert(K, N, M), rand((M, K), 2)
    gives_up(lambda: fp8.shared_expert(x, *w))


@pytest.mark.parametrize("M,N,K", [(4, 512, 2048), (20, 512, 2048), (50, 512, 2048), (100, 256, 1024), (2048, 2048, 512),
                                   (2049, 2047, 144)])
def test_wait_limit_does_not_count_the_kernel_in_front(M, N, K):
    # (in front: a product of 8 CTAs that lets the next one start at once and takes many times the limit)
    deep = 1 << 22
    a, b = torch.zeros(1, deep, dtype=torch.uint8, device="cuda"), torch.zeros(128, deep, dtype=torch.uint8, device="cuda")
    a_s, b_s = torch.ones(1, deep // 128, device="cuda"), torch.ones(1, deep // 128, device="cuda")
    ops = operands(M, N, K, M)
    want = fp8.matmul(*ops)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    fp8.matmul(a, a_s, b, b_s)
    assert fp8.status() == 0
    begin.record()
    fp8.matmul(a, a_s, b, b_s)
    end.record()
    end.synchronize()
    limit = 25  # us, of at least 4 cycles a nanosecond: about 50 at this part's clock
    assert begin.elapsed_time(end) * 1e3 > 10 * limit
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, limit)
    try:
        fp8.matmul(a, a_s, b, b_s)
        got = fp8.matmul(*ops)
        assert fp8.status() == 0
    finally:
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 0)
    assert torch.equal(got, want)


def test_plain_binding():
    # (the calls of the C header as they are, without the checks of fp8 and routing)
    M, K, N = 20, 256, 128
    x, w = rand((M, K), 1), rand((N, K), 2, 0.05)
    new = lambda *shape, dtype: torch.empty(shape, dtype=dtype, device="cuda")
    byte = lambda t: t.view(torch.uint8)
    a, a_s, b, b_s = fp8.quantize(x) + fp8.quantize_weight(w)
    q, s = new(M, K, dtype=torch.uint8), new(M, 2, dtype=torch.float32)
    pkg.moe_w4a16_fp8_quantize(x, BF16, K, M, K, q, s)
    assert torch.equal(q, byte(a)) and torch.equal(s, a_s)
    q, s = new(N, K, dtype=torch.uint8), new(1, 2, dtype=torch.float32)
    pkg.moe_w4a16_fp8_quantize_weight(w, BF16, K, N, K, q, s)
    assert torch.equal(q, byte(b)) and torch.equal(s, b_s)
    q, s = new(M, N, dtype=torch.uint8), new(M, 1, dtype=torch.float32)
    pkg.moe_w4a16_fp8_swiglu_quantize(x, BF16, K, M, N, q, s)
    want = fp8.swiglu_quantize(x)
    assert torch.equal(q, byte(want[0])) and torch.equal(s, want[1])
    out = new(M, N, dtype=torch.float32)
    pkg.moe_w4a16_fp8_matmul(a, K, a_s, b, K, b_s, None, out, F32, M, N, K)
    assert torch.equal(out, fp8.matmul(a, a_s, b, b_s, out_dtype=torch.float32))
    ids, wts = new(M, 8, dtype=torch.int32), new(M, 8, dtype=torch.float32)
    pkg.moe_w4a16_route_scored(x, BF16, K, M, K, 8, pkg.SCORE_SIGMOID, None, 1, 1, 1, True, 1.0, ids, wts)
    want = routing.route_scored(x, 8)
    assert torch.equal(ids, want[0]) and torch.equal(wts, want[1])
    e = expert(K, N, 3)
    want = fp8.shared_expert(x, *e)
    ws = new(pkg.moe_w4a16_shared_expert_workspace_size(M, K, N), dtype=torch.uint8)
    for workspace in (ws, None):
        out = new(M, K, dtype=torch.bfloat16)
        pkg.moe_w4a16_shared_expert(x, *e, None, out, M, K, N, workspace)
        assert torch.equal(out, want)
