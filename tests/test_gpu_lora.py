"""Low-rank adapters of many requests on the GPU against their 64-bit definition.

Tolerance of a value: half a step of the output's type; the second product's r terms (each
of up to three parts) and the addend, summed in fp32 one after another, 3 r / 8 + 8 steps of
2^-23 of their magnitudes (2^-23: matrix units may cut off instead of rounding); and what the
first product's sums of K terms are off by, K / 16 + 24 such steps of both products' terms
(16 or more terms enter a matrix unit's sum at a time; the CUDA cores take 32 at once)."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import MoeW4A16Error, fp8, lora
from oracle import dispatch_oracle as do
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def host(t):
    return None if t is None else t.float().cpu().numpy()


def normal(*shape, seed, by=1.0, dtype=BF16):
    return dev((np.random.default_rng(seed).standard_normal(shape) * by).astype(np.float32)).to(dtype)


def problem(M, K, N, r, L, seed=0):
    x = normal(M, K, seed=seed)
    a, b = normal(L, r, K, seed=seed + 1, by=K ** -0.5), normal(L, N, r, seed=seed + 2, by=r ** -0.5)
    index = np.random.default_rng(seed + 3).integers(-1, L, M).astype(np.int32)
    return x, a, b, index


def check(x, a, b, index, scale=None, add=None, out_dtype=BF16, rows=None, **kw):
    """Rows ``rows`` (default: all) of the call's result against the definition."""
    K, r = x.shape[1], a.shape[1]
    add_before = None if add is None else add.clone()
    got = lora.apply(x, a, b, dev(index), scale=scale, add=add, out_dtype=out_dtype, **kw)
    rows = slice(None) if rows is None else rows
    want, second, both = do.lora(host(x[rows]), host(a), host(b), index[rows], host(scale),
                                 None if add is None else host(add_before[rows]))
    plus = 0.0 if add is None else np.abs(host(add_before[rows]))
    limit = (HALF[got.dtype] * np.abs(want) + (3 * r / 8 + 8) * 2.0 ** -23 * (second + plus) +
             (K / 16 + 24) * 2.0 ** -23 * both)
    over = np.abs(host(got[rows]).astype(np.float64) - want) - limit
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} beyond the limit, by up to {np.nanmax(over)}"
    return got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 129, 300])
@pytest.mark.parametrize("K,N,r,L", [(256, 128, 8, 4), (512, 1000, 16, 32), (1032, 264, 24, 3), (2048, 640, 64, 1),
                                     (776, 72, 128, 5), (7168, 512, 32, 9)])
def test_matches_the_definition(M, K, N, r, L):
    x, a, b, index = problem(M, K, N, r, L, seed=M + K)
    scale = normal(L, seed=7, dtype=F32)
    add = normal(M, N, seed=8, dtype=F32)
    check(x, a, b, index, scale, add)
    check(x, a, b, index, None, add.to(BF16))
    check(x, a, b, index, scale, add.to(BF16), out_dtype=F32)
    check(x, a, b, index, scale, None, out_dtype=F32)


@pytest.mark.parametrize("M", [1, 40, 1100])
@pytest.mark.parametrize("K,N,r", [(1, 1, 1), (33, 77, 3), (100, 130, 12), (257, 250, 8), (264, 41, 5), (40, 8, 127)])
def test_any_size(M, K, N, r):
    x, a, b, index = problem(M, K, N, r, 5, seed=M + K)
    add = normal(M, N, seed=8, dtype=F32)
    rows = None if M < 100 else np.random.default_rng(0).integers(0, M, 64)
    check(x, a, b, index, None, add, rows=rows)
    check(x, a, b, index, None, None, out_dtype=F32, rows=rows)


@pytest.mark.parametrize("M,K,N,r,L", [(700, 512, 384, 16, 6), (1500, 1024, 520, 64, 3), (2049, 776, 264, 40, 40),
                                       (4096, 512, 256, 128, 2), (1025, 2048, 1032, 8, 1000), (5000, 256, 128, 32, 1)])
@pytest.mark.parametrize("spread", ["mixed", "runs", "one", "none"])
def test_many_rows(M, K, N, r, L, spread):
    x, a, b, index = problem(M, K, N, r, L, seed=K)
    if spread == "runs":
        index = np.sort(index)[::-1].copy()
    elif spread == "one":
        index[:] = L - 1
    elif spread == "none":
        index[:] = -1
    rows = np.concatenate([np.arange(20), np.arange(M - 20, M), np.random.default_rng(0).integers(0, M, 100)])
    scale = normal(L, seed=7, dtype=F32)
    for add_type, out_type in ((F32, BF16), (BF16, BF16), (BF16, F32), (None, F32)):
        add = None if add_type is None else normal(M, N, seed=8, dtype=add_type)
        got = check(x, a, b, index, scale, add, out_dtype=out_type, rows=rows)
        if spread == "none" and add is not None:
            assert torch.equal(got, add.to(out_type))


@pytest.mark.parametrize("M", [5, 200, 1300])
def test_in_place_and_rows_without_an_adapter(M):
    x, a, b, index = problem(M, 512, 256, 16, 4)
    index[::3] = -1
    index[1::7] = 4          # no adapter either
    index[2::7] = -2 ** 31
    add = normal(M, 256, seed=9)
    before = add.clone()
    rows = None if M < 300 else np.arange(0, M, 11)
    got = check(x, a, b, index, None, add, rows=rows, out=add)
    assert got is add
    other = lora.apply(x, a, b, dev(index), add=before)
    assert torch.equal(other, add)
    none = torch.from_numpy((index < 0) | (index >= 4)).cuda()
    assert torch.equal(add[none], before[none])
    # rows without an adapter are not touched, nor computed with
    x[none] = float("nan")
    assert torch.equal(lora.apply(x, a, b, dev(index), add=before), add)


@pytest.mark.parametrize("M", [7, 900])
def test_values_that_are_not_numbers_stay_in_their_rows(M):
    x, a, b, index = problem(M, 256, 128, 16, 6)
    index = (np.arange(M) % 6).astype(np.int32)
    x[3, 5] = float("nan")
    x[4, 0] = float("inf")
    a[5, 2, 3] = float("nan")     # an adapter of other requests
    got = lora.apply(x, a, b, dev(index), add=normal(M, 128, seed=4))
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[3] = bad[4] = True
    bad |= dev(index) == 5
    assert got[~bad].isfinite().all() and got[3].isnan().all() and not got[4].isfinite().any()
    assert got[dev(index) == 5].isnan().all()


@pytest.mark.parametrize("M", [6, 900])
def test_strides_and_alignment(M):
    big = normal(2 * M, 700, seed=1)
    for x in (big[:M, 8:520], big[:M, 1:513], big[::2, 16:528], big[M:M + 1, 3:515]):
        m = len(x)
        _, a, b, index = problem(m, 512, 136, 16, 3, seed=m)
        rows = None if m < 100 else np.arange(0, m, 9)
        check(x, a, b, index, None, normal(m, 136, seed=2), rows=rows)
    x, a, b, index = problem(M, 256, 130, 16, 3)
    store = torch.zeros(M * 130 + 1, device="cuda", dtype=BF16)
    out, add = store[1:].view(M, 130), normal(M, 130, seed=3, dtype=F32)
    rows = None if M < 100 else np.arange(0, M, 9)
    check(x, a, b, index, None, add, rows=rows, out=out)
    wide = torch.zeros(a.numel() + 1, device="cuda", dtype=BF16)[1:].view(a.shape).copy_(a)
    check(x, wide, b, index, None, add, rows=rows)


@pytest.mark.parametrize("M", [9, 1200, 2500])
def test_same_bits_other_stream_workspace_and_graphs(M):
    x, a, b, index = problem(M, 1024, 512, 32, 7)
    index, add = dev(index), normal(M, 512, seed=1, dtype=F32)
    first = lora.apply(x, a, b, index, add=add)
    size = lora._workspace_size(M, 1024, 512, 32, 7)
    ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    assert torch.equal(lora.apply(x, a, b, index, add=add, workspace=ws), first)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = lora.apply(x, a, b, index, add=add, stream=s)
    s.synchronize()
    assert torch.equal(other, first)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    for i, g in enumerate(graphs):  # (one with a workspace, one without)
        with torch.cuda.graph(g):
            outs.append(lora.apply(x, a, b, index, add=add, workspace=ws if i else None))
    x.copy_(normal(M, 1024, seed=77))
    index.copy_(torch.randint(-1, 7, (M,), device="cuda", dtype=torch.int32))
    for g in graphs:
        g.replay()
    want = lora.apply(x, a, b, index, add=add)
    for o in outs:
        assert torch.equal(o, want)
    if size > 0:
        with pytest.raises(MoeW4A16Error):
            lora.apply(x, a, b, index, add=add, workspace=ws[:size - 1])


def test_beside_the_8_bit_product():
    M, K, N = 70, 512, 384
    x, a, b, index = problem(M, K, N, 16, 4)
    q, s = fp8.quantize(x)
    w, w_s = fp8.quantize_weight(normal(N, K, seed=5, by=K ** -0.5))
    y = fp8.matmul(q, s, w, w_s, out_dtype=F32)
    check(x, a, b, index, None, y)


def test_no_rows_and_refusals():
    x, a, b, index = problem(6, 64, 40, 8, 3)
    index = dev(index)
    assert lora.apply(x[:0], a, b, index[:0]).shape == (0, 40)
    for call in (lambda: lora.apply(x.float(), a, b, index), lambda: lora.apply(x, a.float(), b, index),
                 lambda: lora.apply(x, a, b[:, :, :7], index), lambda: lora.apply(x, a[0], b, index),
                 lambda: lora.apply(x, a, b, index.long()), lambda: lora.apply(x, a, b, index[:5]),
                 lambda: lora.apply(x, a, b, index, scale=torch.zeros(2, device="cuda")),
                 lambda: lora.apply(x, a, b, index, add=torch.zeros(6, 39, device="cuda")),
                 lambda: lora.apply(x, a, b, index, add=torch.zeros(6, 40, device="cuda", dtype=torch.float16)),
                 lambda: lora.apply(x, a, b, index, out=torch.zeros(5, 40, device="cuda")),
                 lambda: lora.apply(x.t(), a, b, index)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(MoeW4A16Error):
        lora.apply(x, torch.zeros(3, 136, 64, device="cuda", dtype=BF16),
                   torch.zeros(3, 40, 136, device="cuda", dtype=BF16), index)


def test_a_wait_that_gives_up_is_reported():
    import int4_weight_only_moe_gb300 as pkg
    x, a, b, index = problem(1000, 1024, 640, 32, 3)
    add = normal(1000, 640, seed=1)
    want = lora.apply(x, a, b, dev(index), add=add)
    assert fp8.status() == 0
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 1000)
    pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_TEST_WAIT_NEVER_COMPLETES, 1)
    try:
        lora.apply(x, a, b, dev(index), add=add)
        assert fp8.status() == pkg.STATUS_TIMEOUT
    finally:
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_WAIT_LIMIT_US, 0)
        pkg.moe_w4a16_fp8_set_option(pkg.FP8_OPT_TEST_WAIT_NEVER_COMPLETES, 0)
    assert torch.equal(lora.apply(x, a, b, dev(index), add=add), want) and fp8.status() == 0


@pytest.mark.parametrize("M", [5, 900])
@pytest.mark.parametrize("r,K,N", [(8, 256, 128), (24, 264, 136), (16, 256, 128), (3, 33, 20)])
def test_an_infinite_sum_is_infinite(M, r, K, N):
    # positive factors: what the definition makes infinite is +infinity, not NaN
    x, a, b, _ = problem(M, K, N, r, 2)
    x, a, b = x.abs() + 0.25, a.abs() + 0.25, b.abs() + 0.25
    x[1, K - 1] = float("inf")
    got = lora.apply(x, a, b, torch.zeros(M, device="cuda", dtype=torch.int32), add=normal(M, N, seed=1))
    assert (got[1] == float("inf")).all() and got[0].isfinite().all() and got[2:].isfinite().all()
