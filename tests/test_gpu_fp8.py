"""The 8-bit block-scaled operators on the GPU against their float64 definitions.

Tolerances, from the arithmetic:
* quantize / quantize_weight: the scale and the quotient are single 32-bit roundings, as
  in the definition, and so is the e4m3 value: equal.
* swiglu_quantize: h carries an fp32 error (below 1e-5 of it for gates up to 2^5 in
  magnitude); the value kept is h rounded to e4m3 steps: |q s - h| <= 2^-4 |h| + 2^-10 s
  (+ that error), and s within 1e-5.
* matmul: products of e4m3 values are exact; sums of n terms in fp32 err by at most n
  ulp (2^-23) of the sum of magnitudes, with 128 terms to a block and one more per
  block; bf16 outputs by 2^-8 of the result more.
* shared expert: the framework's tolerance of the feed-forward (its bf16 output)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import MoeW4A16Error, fp8
from oracle import ops_oracle as oo
from tests.gpu_helpers import assert_close, bf16_tensor_to_f64, dev

pytestmark = pytest.mark.gpu

ULP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def np64(t):
    return t.float().cpu().numpy().astype(np.float64)


def e4m3(t):
    return oo.e4m3_values(t.view(torch.uint8).cpu().numpy())


def rand(shape, seed, scale=1.0, dtype=torch.bfloat16):
    rng = np.random.default_rng(seed)
    return dev((rng.standard_normal(shape) * scale).astype(np.float32)).to(dtype)


# ----------------------------------------------------------------------------- quantisers


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 7168), (3, 127), (5, 128), (2, 129), (17, 136), (64, 2048), (257, 1000)])
def test_quantize(M, K, dtype):
    x = rand((M, K), M * K, 3.0, dtype)
    q, s = fp8.quantize(x)
    rq, rs = oo.quantize(np64(x))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(e4m3(q), rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (129, 257), (200, 1000), (384, 512)])
def test_quantize_weight(N, K, dtype):
    w = rand((N, K), N + K, 0.02, dtype)
    q, s = fp8.quantize_weight(w)
    rq, rs = oo.quantize_weight(np64(w))
    np.testing.assert_array_equal(s.cpu().numpy(), rs)
    np.testing.assert_array_equal(e4m3(q), rq)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 2048), (7, 130), (33, 136), (300, 256)])
def test_swiglu_quantize(M, N, dtype):
    gu = rand((M, 2 * N), M + N, 4.0, dtype)
    q, s = fp8.swiglu_quantize(gu)
    x = np64(gu)
    h = oo.silu(x[:, :N]) * x[:, N:]
    rs = oo.quantize(h)[1]
    np.testing.assert_allclose(s.cpu().numpy(), rs, rtol=1e-5)
    sp = np.repeat(rs.astype(np.float64), 128, 1)[:, :N]
    bound = (2.0 ** -4 + 2e-5) * np.abs(h) + (2.0 ** -10 + 1e-5) * sp
    assert (np.abs(e4m3(q) * sp - h) <= bound).all()


def test_quantize_ranges_and_special_values():
    x = torch.zeros(10, 256, device="cuda")
    x[1] = 1e-40                                 # subnormal: below the scale's floor
    x[2, 7] = torch.finfo(torch.float32).max
    x[3, :128] = torch.finfo(torch.bfloat16).min
    x[4, 3] = float("nan")
    x[5, 200] = float("inf")
    x[6] = torch.linspace(-1, 1, 256, device="cuda")
    x[7] = 2.0 ** -110 * torch.linspace(-1, 1, 256, device="cuda")
    x[8] = 2.0 ** 110 * torch.linspace(-1, 1, 256, device="cuda")
    x[9, ::2] = -0.0
    for t in (x, x.to(torch.bfloat16)):
        q, s = fp8.quantize(t)
        q, s = e4m3(q), s.cpu().numpy()
        fine = [0, 1, 2, 3, 6, 7, 8, 9]
        if t.dtype == torch.bfloat16:
            fine.remove(2)                       # (rounds to infinity in bf16)
        rq, rs = oo.quantize(np64(t)[fine])
        np.testing.assert_array_equal(s[fine], rs)
        np.testing.assert_array_equal(q[fine], rq)
        assert np.isnan(s[4, 0]) and np.isnan(q[4, :128]).all() and not np.isnan(q[4, 128:]).any()
        assert np.isinf(s[5, 1]) and np.isnan(q[5, 200]) and not q[5, :200].any()


def test_quantize_strides_alignment_out_and_empty():
    big = rand((50, 640), 3)
    for part in (big[:, 1:300], big[:, 8:520], big[::3, :256], big[7:8, 3:131]):
        q, s = fp8.quantize(part)
        rq, rs = oo.quantize(np64(part))
        np.testing.assert_array_equal(e4m3(q), rq)
        np.testing.assert_array_equal(s.cpu().numpy(), rs)
        wq, ws = fp8.quantize_weight(part)
        rq, rs = oo.quantize_weight(np64(part))
        np.testing.assert_array_equal(e4m3(wq), rq)
        np.testing.assert_array_equal(ws.cpu().numpy(), rs)
    raw = torch.zeros(50 * 256 + 1, dtype=torch.uint8, device="cuda")
    q, s = fp8.quantize(big[:, :256].contiguous(), q=raw[1:].view(50, 256))  # odd address
    np.testing.assert_array_equal(e4m3(q), oo.quantize(np64(big[:, :256]))[0])
    assert raw[0] == 0
    q, s = fp8.quantize(big[:0])
    assert q.shape == (0, 640) and s.shape == (0, 5)


def test_quantize_beyond_32_bit_offsets():
    M, K = 310_000, 7168  # 2.2e9 values
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-3:] = rand((3, K), 4)
    q, s = fp8.quantize(x)
    rq, rs = oo.quantize(np64(x[-3:]))
    np.testing.assert_array_equal(e4m3(q[-3:]), rq)
    np.testing.assert_array_equal(s[-3:].cpu().numpy(), rs)


# -------------------------------------------------------------------------------- product


def operands(M, N, K, seed):
    a, a_s = fp8.quantize(rand((M, K), seed, 2.0))
    b, b_s = fp8.quantize_weight(rand((N, K), seed + 1, 0.05))
    return a, a_s, b, b_s


def check_product(got, a, a_s, b, b_s, add=None):
    K = a.shape[1]
    ref, mag = oo.matmul(e4m3(a), a_s.cpu().numpy(), e4m3(b), b_s.cpu().numpy(), None if add is None else np64(add))
    tol = (min(K, 128) + -(-K // 128) + 4) * ULP * (mag + (0.0 if add is None else np.abs(np64(add))))
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    err = np.abs(np64(got) - ref)
    assert (err <= tol).all(), float((err - tol).max())


SHAPES = [(1, 1, 1), (1, 1, 16), (3, 5, 7), (1, 128, 128), (1, 4096, 7168), (2, 130, 17), (4, 256, 512), (9, 7168, 2048),
          (16, 128, 384), (17, 129, 144), (31, 1000, 1936), (33, 640, 128), (64, 4096, 640), (65, 256, 1024),
          (90, 512, 2048), (128, 128, 128), (129, 257, 272), (200, 384, 7168), (257, 96, 400), (300, 1000, 1936),
          (513, 1024, 384), (1030, 2048, 512), (2048, 768, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(M, N, K):
    ops = operands(M, N, K, M + N + K)
    check_product(fp8.matmul(*ops, out_dtype=torch.float32), *ops)
    add = rand((M, N), 5)
    check_product(fp8.matmul(*ops, add=add), *ops, add=add)


@pytest.mark.parametrize("M", [1, 2, 8, 15, 16, 24, 32, 48, 63, 72, 96, 127, 136, 160, 192, 250, 256, 320, 511, 600])
def test_product_over_batch_sizes(M):
    # (every variant, and the borders between them)
    for N, K in ((256, 384), (1152, 2048)):
        ops = operands(M, N, K, 7 * M)
        check_product(fp8.matmul(*ops, out_dtype=torch.float32), *ops)


def test_product_strides_and_alignment():
    raw_a, raw_b = rand((70, 2000), 1), rand((300, 2000), 2, 0.05)
    full_a = fp8.quantize(raw_a)[0].view(torch.uint8)
    full_b = fp8.quantize(raw_b)[0].view(torch.uint8)
    for off, K, step in ((0, 512, 1), (16, 512, 1), (16, 500, 1), (1, 512, 1), (7, 129, 1), (0, 1040, 2)):
        a, b = full_a[::step, off:off + K], full_b[:, off:off + K]
        M, N, Kb = a.shape[0], b.shape[0], -(-K // 128)
        a_s = dev(np.random.default_rng(K).uniform(0.5, 2, (M, Kb)).astype(np.float32))
        b_s = dev(np.random.default_rng(off).uniform(0.5, 2, (-(-N // 128), Kb)).astype(np.float32))
        check_product(fp8.matmul(a, a_s, b, b_s, out_dtype=torch.float32), a, a_s, b, b_s)
    # outputs and addends that are not at the start of an allocation
    ops = operands(70, 300, 512, 3)
    for off in (1, 3, 4):
        buf = torch.zeros(70 * 300 + 8, dtype=torch.bfloat16, device="cuda")
        out = buf[off:off + 70 * 300].view(70, 300)
        add = rand(70 * 300 + 8, 8)[8 - off:8 - off + 70 * 300].view(70, 300)
        check_product(fp8.matmul(*ops, add=add, out=out), *ops, add=add)
        assert not buf[:off].any() and not buf[off + 70 * 300:].any()


@pytest.mark.parametrize("M", [33, 40, 49, 64, 65])
def test_product_of_33_to_64_rows(M):
    for N, K in ((130, 144), (700, 640), (1152, 2048), (7168, 256)):
        ops = operands(M, N, K, 3 * M)
        add = rand((M, N), 5)
        check_product(fp8.matmul(*ops, add=add), *ops, add=add)
    w, x = expert(1024, 384, M), rand((M, 1024), 2)
    assert_close(bf16_tensor_to_f64(fp8.shared_expert(x, *w)), expert_reference(x, w), "shared expert")


@pytest.mark.parametrize("M,N,K", [(65535 * 128 + 5, 1, 16), (1, 65535 * 64 + 5, 8)])
def test_product_with_more_tiles_than_a_grid_dimension(M, N, K):
    # (small whole numbers: every sum is exact)
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randint(-4, 5, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-4, 5, (N, K), generator=g, device="cuda").float()
    a_s = torch.ones(M, 1, device="cuda")
    b_s = torch.full(((N + 127) // 128, 1), 0.5, device="cuda")
    out = fp8.matmul(a.to(torch.float8_e4m3fn), a_s, b.to(torch.float8_e4m3fn), b_s, out_dtype=torch.float32)
    assert torch.equal(out.view(-1), (a * b).sum(1) * 0.5)


@pytest.mark.parametrize("M,N", [(3, 256), (90, 700), (600, 512)])
def test_add_in_place(M, N):
    ops = operands(M, N, 640, 9)
    out = rand((M, N), 4)
    add = out.clone()
    assert fp8.matmul(*ops, add=out, out=out) is out
    check_product(out, *ops, add=add)


@pytest.mark.parametrize("M", [2, 40, 300])
def test_scales_of_wide_range_zero_and_nan(M):
    N, K = 200, 512
    ops = operands(M, N, K, 12)
    a, _, b, _ = ops
    rng = np.random.default_rng(M)
    a_s = dev(np.exp2(rng.integers(-40, 40, (M, 4))).astype(np.float32))
    b_s = dev(np.exp2(rng.integers(-40, 40, (2, 4))).astype(np.float32))
    a_s[0] = 0.0
    check_product(fp8.matmul(a, a_s, b, b_s, out_dtype=torch.float32), a, a_s, b, b_s)
    clean = fp8.matmul(*ops, out_dtype=torch.float32)
    bad = a.view(torch.uint8).clone()
    bad[1, 300] = 0x7F  # NaN in one row
    got = fp8.matmul(bad, *ops[1:], out_dtype=torch.float32)
    assert got[1].isnan().all()
    keep = [i for i in range(M) if i != 1]
    assert torch.equal(got[keep], clean[keep])
    bad = b.view(torch.uint8).clone()
    bad[130, 0] = 0xFF  # ... and in one column
    got = fp8.matmul(a, ops[1], bad, ops[3], out_dtype=torch.float32)
    assert got[:, 130].isnan().all()
    assert torch.equal(got[:, :130], clean[:, :130]) and torch.equal(got[:, 131:], clean[:, 131:])


def test_repeats_are_equal_and_other_stream():
    for M in (1, 40, 200, 700):
        ops = operands(M, 1000, 2048, M)
        first = fp8.matmul(*ops)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        other = fp8.matmul(*ops, stream=s)
        for _ in range(5):
            assert torch.equal(fp8.matmul(*ops), first)
        s.synchronize()
        assert torch.equal(other, first)


def test_empty():
    a, a_s, b, b_s = operands(4, 64, 256, 0)
    assert fp8.matmul(a[:0], a_s[:0], b, b_s).shape == (0, 64)
    assert fp8.matmul(a, a_s, b[:0], b_s[:0]).shape == (4, 0)


@pytest.mark.slow
def test_output_beyond_32_bit_offsets():
    M, N, K = 550_000, 4000, 128  # 2.2e9 outputs
    ops = operands(M, N, K, 1)
    out = fp8.matmul(*ops)
    tail = [ops[0][-300:].contiguous(), ops[1][-300:].contiguous(), ops[2], ops[3]]
    check_product(out[-300:], *tail)


def test_refusals():
    a, a_s, b, b_s = operands(4, 64, 256, 0)
    with pytest.raises(ValueError):
        fp8.matmul(a, a_s, b[:, :128], b_s)
    with pytest.raises(ValueError):
        fp8.matmul(a, a_s[:, :1], b, b_s)
    with pytest.raises(ValueError):
        fp8.matmul(a, a_s, b, b_s, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fp8.matmul(a, a_s, b, b_s, add=torch.zeros(4, 64, device="cuda"))
    with pytest.raises(ValueError):
        fp8.matmul(a.view(torch.uint8).t(), a_s, b, b_s)
    with pytest.raises(ValueError):
        fp8.quantize(torch.zeros(4, 64, device="cuda", dtype=torch.float16))
    with pytest.raises(MoeW4A16Error):
        fp8.quantize(torch.zeros(4, 0, device="cuda"))


# -------------------------------------------------------------------------- shared expert


def expert(K, N, seed):
    w1, w1_s = fp8.quantize_weight(rand((2 * N, K), seed, K ** -0.5))
    w2, w2_s = fp8.quantize_weight(rand((K, N), seed + 1, N ** -0.5))
    return w1, w1_s, w2, w2_s


def expert_reference(x, w, add=None):
    w1, w1_s, w2, w2_s = w
    return oo.shared_expert(np64(x), e4m3(w1), w1_s.cpu().numpy(), e4m3(w2), w2_s.cpu().numpy(),
                            None if add is None else np64(add))


@pytest.mark.parametrize("M,K,N", [(1, 128, 128), (1, 7168, 2048), (4, 512, 256), (17, 256, 384), (70, 1024, 640),
                                   (130, 384, 128), (300, 512, 1152), (515, 640, 512)])
def test_shared_expert(M, K, N):
    w = expert(K, N, M)
    x, add = rand((M, K), 2), rand((M, K), 3)
    assert_close(bf16_tensor_to_f64(fp8.shared_expert(x, *w)), expert_reference(x, w), "shared expert")
    want = expert_reference(x, w, add)
    out = fp8.shared_expert(x, *w, add=add)
    assert_close(bf16_tensor_to_f64(out), want, "shared expert + routed")
    mine = add.clone()
    fp8.shared_expert(x, *w, add=mine, out=mine)  # in place
    assert torch.equal(mine, out)


def test_shared_expert_workspace_stream_and_empty():
    from int4_weight_only_moe_gb300 import moe_w4a16_shared_expert_workspace_size
    K, N, M = 256, 128, 9
    w = expert(K, N, 1)
    x = rand((M, K), 2)
    want = fp8.shared_expert(x, *w)
    ws = torch.full((moe_w4a16_shared_expert_workspace_size(M, K, N),), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(fp8.shared_expert(x, *w, workspace=ws), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = fp8.shared_expert(x, *w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    assert fp8.shared_expert(x[:0], *w).shape == (0, K)
    with pytest.raises(MoeW4A16Error):
        fp8.shared_expert(x, *w, workspace=ws[:-1])


def test_shared_expert_takes_its_workspace_from_the_pool_or_torch():
    # (below and above the pool's limit; calls in flight on two streams do not share it)
    from int4_weight_only_moe_gb300 import moe_w4a16_shared_expert_workspace_size as size
    K, N = 2048, 256
    w = expert(K, N, 5)
    for M in (64, 9000):
        assert (size(M, K, N) > fp8._POOL_BYTES) == (M == 9000)
        x, y = rand((M, K), 1), rand((M, K), 2)
        ws = torch.empty(size(M, K, N), dtype=torch.uint8, device="cuda")
        want = [fp8.shared_expert(t, *w, workspace=ws).clone() for t in (x, y)]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = [[fp8.shared_expert(t, *w, stream=s) for t, s in zip((x, y), streams)] for _ in range(8)]
        torch.cuda.synchronize()
        for pair in got:
            assert torch.equal(pair[0], want[0]) and torch.equal(pair[1], want[1])


def test_first_call_of_a_process_may_be_captured():
    code = """
import torch
from int4_weight_only_moe_gb300 import fp8
M, K, N = 100, 1024, 512
bytes_ = lambda *n: torch.randint(0, 100, n, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
h = torch.randn(M, K, device="cuda").bfloat16()
w = (bytes_(2 * N, K), torch.rand(8, 8, device="cuda") * 0.01, bytes_(K, N), torch.rand(8, 4, device="cuda") * 0.01)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = fp8.shared_expert(h, *w)
g.replay()
torch.cuda.synchronize()
assert torch.equal(y, fp8.shared_expert(h, *w)) and fp8.status() == 0 and y.isfinite().all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_shared_expert_replays_from_a_cuda_graph():
    K, N = 512, 256
    w = expert(K, N, 4)
    for M in (2, 200):
        x, out = rand((M, K), 1), torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        fp8.shared_expert(x, *w, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fp8.shared_expert(x, *w, out=out)
        x.copy_(rand((M, K), 2))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fp8.shared_expert(x, *w))


# ------------------------------------------------------------------------------- give-up


@pytest.mark.parametrize("M,N,K", [(4, 512, 2048), (20, 512, 2048), (50, 512, 2048), (100, 256, 1024), (1200, 2048, 1024)])
def test_wait_limit_gives_up_cleanly(M, N, K):
    """A wait that nothing completes runs out: the call returns, the status says so, and the
    next call is right (one size for each kernel)."""
    import int4_weight_only_moe_gb300 as pkg
    ops = operands(M, N, K, M)
    x, w = rand((M, K), 1), expert(K, N, 2)
    want, whole = fp8.matmul(*ops), fp8.shared_expert(x, *w)
    assert fp8.status() == 0
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 1000)
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_TEST_WAIT_NEVER_COMPLETES, 1)
    try:
        fp8.matmul(*ops)
        assert fp8.status() == pkg.STATUS_TIMEOUT
        fp8.shared_expert(x, *w)
        assert fp8.status() == pkg.STATUS_TIMEOUT
    finally:
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_TEST_WAIT_NEVER_COMPLETES, 0)
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 0)
    assert fp8.status() == 0
    assert torch.equal(fp8.matmul(*ops), want) and torch.equal(fp8.shared_expert(x, *w), whole)
    assert fp8.status() == 0
