"""Tokens sorted by expert and back, the gradients of both, on the GPU against their 64-bit
definitions. Whole numbers and moved rows have to be equal.

Tolerances. HALF is half a step of the output's type relative to the value. A sum of n fp32
fused products, in any order, is off by at most n 2^-24 of the sum of its terms' magnitudes;
combine adds topk products and an addend, a gradient of a weight K products: at most
ceil(K / 128) + 8 of them one after another in a thread (128 share a token), 5 + 8 additions across the CTA, the
product's rounding taken up by the fused operation; two more for what was rounded before."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import MoeW4A16Error, dispatch
from oracle import dispatch_oracle as do
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def host(t):
    return t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def some_ids(M, topk, E, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(max(E, topk))[:topk] % E for _ in range(M)]) if M else np.zeros((0, topk))
    ids = np.where(rng.random((M, topk)) < 0.5, (ids * ids) % E, ids)  # some experts busier than others
    return np.where(rng.random((M, topk)) < drop, rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], (M, topk)), ids).astype(np.int32)


def same_order(got, want):
    for g, w in zip(got, want):
        np.testing.assert_array_equal(host(g), w)


SIZES = [(1, 1, 1), (1, 8, 384), (3, 2, 5), (4, 8, 384), (31, 1, 7), (90, 8, 384), (128, 8, 64), (129, 8, 1024),
         (333, 6, 160), (700, 8, 1), (511, 32, 33), (2049, 2, 1000), (4097, 1, 3), (3000, 12, 384)]


@pytest.mark.parametrize("M,topk,E", SIZES)
@pytest.mark.parametrize("block", [1, 3, 16, 128])
def test_sort(M, topk, E, block):
    for drop in (0.0, 0.3, 1.0):
        ids = some_ids(M, topk, E, M + E, drop)
        same_order(dispatch.sort(dev(ids), E, block), do.order(ids, E, block))


def test_sort_same_expert_for_all():
    for M, topk, E in ((600, 8, 384), (5000, 3, 2)):
        ids = np.full((M, topk), E - 1, np.int32)
        same_order(dispatch.sort(dev(ids), E, 16), do.order(ids, E, 16))


def test_sort_a_part_of_the_experts():
    ids = some_ids(500, 8, 384, 3, 0.1)
    for begin, end in ((0, 96), (96, 200), (383, 384), (0, 384)):
        got = dispatch.sort(dev(ids), 384, 16, expert_range=(begin, end))
        same_order(got, do.order(ids, end - begin, 16, begin))


def test_sort_of_no_tokens_and_long_lists():
    got = dispatch.sort(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 9, 16)
    assert got.offsets.tolist() == [0] * 10 and got.slots.numel() == 0
    ids = torch.randint(0, 384, (300_001, 8), dtype=torch.int32, device="cuda")
    got = dispatch.sort(ids, 384, 128)
    flat = ids.view(-1).long()
    key, by = torch.sort(flat, stable=True)
    counts = torch.bincount(flat, minlength=384)
    padded = (counts + 127) // 128 * 128
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    row = offsets[key] + torch.arange(flat.numel(), device="cuda") - (counts.cumsum(0) - counts)[key]
    assert torch.equal(got.offsets.long(), offsets)
    position = torch.empty_like(row)
    position[by] = row
    assert torch.equal(got.position.view(-1).long(), position)
    slots = torch.full((got.slots.numel(),), -1, device="cuda")
    slots[row] = by
    assert torch.equal(got.slots.long(), slots)


# ------------------------------------------------------------------------------ gather


@pytest.mark.parametrize("M,topk,E,block,K", [
    (1, 1, 1, 1, 1), (1, 8, 384, 1, 7168), (4, 8, 384, 128, 7168), (3, 3, 5, 2, 33), (17, 4, 12, 16, 1000),
    (90, 8, 384, 1, 257), (333, 6, 160, 16, 640), (1000, 8, 64, 128, 130), (2, 32, 40, 4, 20000), (515, 2, 7, 1, 24)])
@pytest.mark.parametrize("dtype", [F32, BF16, torch.float8_e4m3fn, torch.uint8])
@pytest.mark.parametrize("call", ["gather", "sort_gather"])
def test_gather(M, topk, E, block, K, dtype, call):
    ids = some_ids(M, topk, E, M + K, 0.2)
    x = torch.randint(0, 100, (M, K), device="cuda", dtype=torch.uint8)
    x = x.view(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)
    cap = dispatch.rows(M, topk, E, block)
    out = torch.full((cap, K), 101, device="cuda", dtype=torch.uint8)
    out = out.view(dtype) if dtype == torch.float8_e4m3fn else out.to(dtype)
    before = out.clone()
    want_order = do.order(ids, E, block)
    if call == "gather":
        order = dispatch.Order(*map(dev, want_order))
        got = dispatch.gather(x, order, out=out)
    else:
        got, order = dispatch.sort_gather(x, dev(ids), E, block, out=out)
        same_order(order, want_order)
    assert got is out
    want = do.gather(host(x.float()), want_order[0], want_order[1], topk, host(before.float()))
    np.testing.assert_array_equal(host(out.float()), want)


def test_gather_strided_and_unaligned_rows():
    ids = some_ids(60, 4, 9, 5)
    order = dispatch.sort(dev(ids), 9, 4)
    o = [host(t) for t in order]
    big = torch.randn(121, 700, device="cuda")
    for dtype in (F32, BF16):
        t = big.to(dtype)
        for x in (t[:60, 1:600], t[:60, 4:604], t[1::2, 8:520], t[:60, 3:4]):
            out = torch.zeros(order.slots.numel(), x.shape[1], device="cuda", dtype=dtype)
            want = do.gather(host(x), o[0], o[1], 4, host(out))
            np.testing.assert_array_equal(host(dispatch.gather(x, order, out=out)), want)
            np.testing.assert_array_equal(host(dispatch.sort_gather(x, dev(ids), 9, 4, out=out)[0]), want)


def test_gather_moves_every_bit_pattern():
    bits = torch.arange(-2 ** 15, 2 ** 15, device="cuda", dtype=torch.int32).to(torch.int16).view(BF16).view(64, 1024)
    ids = some_ids(64, 2, 8, 1)
    rows, order = dispatch.sort_gather(bits, dev(ids), 8)
    want = bits.view(torch.int16)[(order.slots // 2).long()]
    assert torch.equal(rows.view(torch.int16), want)


def test_gather_beyond_32_bit_offsets():
    M, topk, K = 40_000, 8, 7168  # 2.3e9 values
    ids = torch.randint(0, 16, (M, topk), dtype=torch.int32, device="cuda")
    x = torch.randn(M, K, device="cuda", dtype=BF16)
    rows, order = dispatch.sort_gather(x, ids, 16)
    at = torch.cat([torch.arange(0, 40, device="cuda"), torch.arange(M * topk - 40, M * topk, device="cuda")])
    assert torch.equal(rows[at], x[(order.slots[at] // topk).long()])
    w = torch.rand(M, topk, device="cuda")
    out = dispatch.combine(rows, w, order)  # every row is the token's own
    for part in (slice(0, 64), slice(M - 64, M)):
        want = x[part].double() * w[part].double().sum(1, keepdim=True)
        # (nine roundings of 2^-24 of a sum of non-negative multiples, and the output's)
        assert ((out[part].double() - want).abs() <= (2.0 ** -8 + 10 * 2.0 ** -24) * want.abs()).all()
    dy, dw = dispatch.combine_backward(x, rows, w, order)
    r = at
    t = (order.slots[r] // topk).long()
    want = w.view(-1)[order.slots[r].long()].double()[:, None] * x[t].double()
    assert ((dy[r].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()


# ------------------------------------------------------------------------------ combine


def close(got, want, limit):
    got = host(got).astype(np.float64)
    assert got.shape == want.shape
    over = np.abs(got - want) - limit
    assert (over <= 0).all(), f"{(over > 0).sum()} of {over.size} beyond the limit, by up to {np.nanmax(over)}"


COMBINE = [(1, 1, 1, 1, 1), (1, 8, 384, 1, 7168), (4, 8, 384, 16, 2048), (90, 8, 384, 1, 1000), (33, 3, 5, 4, 77),
           (333, 6, 64, 1, 256), (7, 32, 40, 1, 520), (129, 9, 12, 128, 64), (2, 17, 3, 1, 9000)]


@pytest.mark.parametrize("M,topk,E,block,K", COMBINE)
@pytest.mark.parametrize("y_type", [F32, BF16])
@pytest.mark.parametrize("out_type", [F32, BF16])
@pytest.mark.parametrize("weighted,added", [(True, True), (True, False), (False, False)])
def test_combine(M, topk, E, block, K, y_type, out_type, weighted, added):
    ids = some_ids(M, topk, E, M * K, 0.15)
    order = dispatch.sort(dev(ids), E, block)
    y = torch.randn(order.slots.numel(), K, device="cuda").to(y_type)
    w = torch.randn(M, topk, device="cuda") if weighted else None
    add = torch.randn(M, K, device="cuda").to(out_type) if added else None
    args = (host(y), None if w is None else host(w), host(order.position), None if add is None else host(add))
    limit = HALF[out_type] * np.abs(do.combine(*args)) + (topk + 2) * 2.0 ** -24 * do.combine_size(*args)
    if weighted:
        got = dispatch.combine(y, w, order, add=add, out_dtype=out_type)
    else:
        got = dispatch.gather_backward(y, order, out_dtype=out_type)
    assert got.dtype == out_type
    close(got, do.combine(*args), limit)
    if added:
        again = dispatch.combine(y, w, order, add=add, out=add)
        assert again is add and torch.equal(again, got)


def test_combine_reads_nothing_of_rows_that_are_no_choices():
    ids = np.array([[0, 1], [1, -1], [-1, -1]], np.int32)
    order = dispatch.sort(dev(ids), 3, 4)
    y = torch.full((order.slots.numel(), 64), float("nan"), device="cuda", dtype=BF16)
    for i, r in enumerate(host(order.position).reshape(-1)):
        if r >= 0:
            y[r] = float(i + 1)
    w = torch.full((3, 2), float("inf"), device="cuda")
    w[0], w[1, 0] = 1.0, 2.0
    got = dispatch.combine(y, w, order)
    assert got[0].eq(3.0).all() and got[1].eq(6.0).all() and got[2].eq(0.0).all()
    g = torch.ones(3, 64, device="cuda", dtype=BF16)
    dy, dw = dispatch.combine_backward(g, y, w, order, dy=torch.full_like(y, 5.0))
    assert torch.isfinite(dw).all() and dw.tolist() == [[64.0, 128.0], [192.0, 0.0], [0.0, 0.0]]
    assert dy[:8].isfinite().all() and dy[8:].eq(5.0).all()


def test_combine_carries_infinities_and_nans_of_its_own_rows_only():
    ids = some_ids(8, 2, 4, 2)
    order = dispatch.sort(dev(ids), 4)
    y = torch.randn(16, 40, device="cuda")
    y[int(order.position[3, 1])] = float("inf")
    y[int(order.position[5, 0])] = float("nan")
    got = dispatch.combine(y, torch.ones(8, 2, device="cuda"), order)
    assert got[3].isinf().all() and got[5].isnan().all()
    assert got[[0, 1, 2, 4, 6, 7]].isfinite().all()


@pytest.mark.parametrize("M,topk,E,block,K", COMBINE)
@pytest.mark.parametrize("y_type", [F32, BF16])
@pytest.mark.parametrize("g_type", [F32, BF16])
def test_combine_backward(M, topk, E, block, K, y_type, g_type):
    ids = some_ids(M, topk, E, M + 3 * K, 0.15)
    order = dispatch.sort(dev(ids), E, block)
    y = torch.randn(order.slots.numel(), K, device="cuda").to(y_type)
    g = torch.randn(M, K, device="cuda").to(g_type)
    w = torch.randn(M, topk, device="cuda")
    before = torch.full_like(y, 7.0)
    dy, dw = dispatch.combine_backward(g, y, w, order, dy=before.clone())
    want, want_w, size = do.combine_backward(host(g), host(y), host(w), *map(host, order), host(before))
    close(dy, want, (HALF[y_type] + (2.0 ** -23 if y_type == BF16 else 0.0)) * np.abs(want))
    close(dw, want_w, (-(-K // 128) + 8 + 13 + 2) * 2.0 ** -24 * size)


def test_gradients_against_differences():
    # combine is linear in y and in w: differences of any width are exact but for roundings
    ids = some_ids(20, 4, 6, 8, 0.1)
    order = dispatch.sort(dev(ids), 6, 4)
    R = order.slots.numel()
    y, w, g = torch.randn(R, 48, device="cuda"), torch.randn(20, 4, device="cuda"), torch.randn(20, 48, device="cuda")
    dy, dw = dispatch.combine_backward(g, y, w, order, dy=torch.zeros_like(y))
    loss = lambda y, w: (dispatch.combine(y, w, order).double() * g.double()).sum()  # noqa: E731
    for seed in range(4):
        torch.manual_seed(seed)
        ey, ew = torch.randn_like(y), torch.randn_like(w)
        # (960 outputs of size about 10, each off by 6 2^-24 of that: below 960 * 10 * 6 * 2^-24 = 3.4e-3)
        assert abs(float(loss(y + ey, w) - loss(y, w)) - float((dy.double() * ey.double()).sum())) < 7e-3
        assert abs(float(loss(y, w + ew) - loss(y, w)) - float((dw.double() * ew.double()).sum())) < 7e-3
    x, dr = torch.randn(20, 48, device="cuda"), torch.randn(R, 48, device="cuda")
    rows = dispatch.gather(x, order, out=torch.zeros(R, 48, device="cuda"))
    dx = dispatch.gather_backward(dr, order)
    dr[int(order.offsets[-1]):] = 0
    # (an adjoint pair: both sides sum the same products; 20 * 4 * 48 of size 1, 5 roundings each)
    assert abs(float((rows.double() * dr.double()).sum() - (x.double() * dx.double()).sum())) < 3840 * 5 * 2.0 ** -24 * 4


# ------------------------------------------------------------------------------ together


def test_same_bits_every_run_other_stream_and_graph():
    M, topk, E, K = 257, 8, 96, 1024
    x = torch.randn(M, K, device="cuda", dtype=BF16)
    ids, w = dev(some_ids(M, topk, E, 4)), torch.rand(M, topk, device="cuda")

    def chain(stream=None):
        rows, order = dispatch.sort_gather(x, ids, E, 16, stream=stream)
        out = dispatch.combine(rows, w, order, stream=stream)
        dy, dw = dispatch.combine_backward(x, rows, w, order, stream=stream)
        n = dispatch.gather_backward(dy, order, stream=stream)
        return out, dw, n

    first = chain()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    second = chain(s)
    s.synchronize()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = chain()
    x.copy_(torch.randn(M, K, device="cuda", dtype=BF16))
    ids.copy_(dev(some_ids(M, topk, E, 5)))
    graph.replay()
    fourth = chain()
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    for a, b in zip(third, fourth):
        assert torch.equal(a, b)


def test_no_tokens():
    order = dispatch.sort(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 9)
    x = torch.zeros(0, 64, device="cuda", dtype=BF16)
    assert dispatch.gather(x, order).shape == (0, 64)
    assert dispatch.combine(x, torch.zeros(0, 4, device="cuda"), order).shape == (0, 64)
    dy, dw = dispatch.combine_backward(x, x.clone(), torch.zeros(0, 4, device="cuda"), order)
    assert dy.shape == (0, 64) and dw.shape == (0, 4)


def test_positions_out_of_range_are_nobodys():
    order = dispatch.sort(dev(some_ids(10, 2, 4, 1)), 4)
    wrong = dispatch.Order(order.offsets, order.slots, order.position.clone())
    wrong.position[0, 0], wrong.position[1, 1] = 2 ** 30, -7
    y, w = torch.randn(20, 32, device="cuda"), torch.rand(10, 2, device="cuda")
    ref = w.clone()
    ref[0, 0] = ref[1, 1] = 0.0
    assert torch.equal(dispatch.combine(y, w, wrong), dispatch.combine(y, ref, order))
    _, dw = dispatch.combine_backward(torch.randn(10, 32, device="cuda"), y, w, wrong)
    assert dw[0, 0] == 0 and dw[1, 1] == 0
    dispatch.gather(torch.randn(10, 32, device="cuda"), wrong)
    torch.cuda.synchronize()


def test_refusals():
    ids = dev(some_ids(6, 2, 4, 1))
    order = dispatch.sort(ids, 4, 2)
    x = torch.zeros(6, 32, device="cuda", dtype=BF16)
    w, y = torch.zeros(6, 2, device="cuda"), torch.zeros(order.slots.numel(), 32, device="cuda", dtype=BF16)
    for call in (lambda: dispatch.sort(ids.long(), 4), lambda: dispatch.sort(ids, 0), lambda: dispatch.sort(ids, 1025),
                 lambda: dispatch.sort(ids, 4, 0), lambda: dispatch.sort(ids.t(), 4), lambda: dispatch.sort(ids[0], 4),
                 lambda: dispatch.sort(ids, 4, expert_range=(2, 2)), lambda: dispatch.sort(ids, 4, expert_range=(2, 5)),
                 lambda: dispatch.gather(x[:5], order), lambda: dispatch.gather(x.double(), order),
                 lambda: dispatch.gather(x.t(), order), lambda: dispatch.gather(x, order, out=y[:-1]),
                 lambda: dispatch.gather(x, dispatch.Order(order.offsets, order.slots[:-1], order.position)),
                 lambda: dispatch.sort_gather(x[:5], ids, 4), lambda: dispatch.combine(y[:-1], w, order),
                 lambda: dispatch.combine(y, w[:, :1], order), lambda: dispatch.combine(y, w, order, add=x.float()),
                 lambda: dispatch.combine(y, w.double(), order), lambda: dispatch.combine_backward(x, y[:-1], w, order),
                 lambda: dispatch.combine_backward(x[:, :31], y, w, order),
                 lambda: dispatch.combine_backward(x, y.half(), w, order)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(MoeW4A16Error):
        dispatch.combine_backward(x, y, w, order, dy=y)
