"""Order, gather, combine, their gradients, the router's gradient and the low-rank adapters
without a GPU: the definitions on values known by hand, and the refusals of the C entries."""
import ctypes

import numpy as np
import pytest

from oracle import dispatch_oracle as do

OK, INVALID, SHAPE, WORKSPACE = 0, -1, -2, -3
F32, BF16, E4M3 = 0, 1, 2


def test_order_by_hand():
    ids = np.array([[2, 0], [0, 5], [2, -1]], np.int32)
    offsets, slots, position = do.order(ids, 3, 2)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert slots.tolist() == [1, 2, 0, 4] + [-1] * 5
    assert position.tolist() == [[2, 0], [1, -1], [3, -1]]
    offsets, slots, position = do.order(ids, 2, 4, begin=2)
    assert offsets.tolist() == [0, 4, 4] and slots.tolist()[:4] == [0, 4, -1, -1]
    assert position.tolist() == [[0, -1], [-1, -1], [1, -1]]


def test_rows_by_hand():
    ids = np.array([[1, 0], [1, -1]], np.int32)
    offsets, slots, position = do.order(ids, 2, 2)
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    rows = do.gather(x, offsets, slots, 2, np.full((len(slots), 2), 9.0))
    assert rows.tolist() == [[1, 2], [0, 0], [1, 2], [3, 4], [9, 9], [9, 9]]
    w = np.array([[0.5, 2.0], [3.0, 7.0]])
    assert do.combine(rows, w, position, np.ones((2, 2))).tolist() == [[3.5, 6], [10, 13]]
    dy, dw, _ = do.combine_backward(x, rows, w, offsets, slots, position, np.full((len(slots), 2), 9.0))
    assert dw.tolist() == [[5, 5], [25, 0]] and dy.tolist() == [[2, 4], [0, 0], [0.5, 1], [9, 12], [9, 9], [9, 9]]


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_backward_is_the_derivative(scoring, renormalize):
    rng = np.random.default_rng(0)
    l, ids, g = rng.standard_normal((3, 9)), np.array([[0, 4, 8], [1, 2, 3], [5, 0, 7]]), rng.standard_normal((3, 3))
    d, _ = do.route_backward(g, l, ids, scoring, renormalize, 2.5)
    for e in range(9):
        h = np.zeros_like(l)
        h[:, e] = 1e-6
        up, down = (do.route_weights(l + s * h, ids, scoring, renormalize, 2.5) for s in (1, -1))
        np.testing.assert_allclose(d[:, e], ((up - down) * g).sum(1) / 2e-6, atol=1e-8)


def test_lora_by_hand():
    x, a = np.array([[1.0, 2.0], [3.0, 4.0]]), np.array([[[1.0, 1.0]], [[0.0, 2.0]]])
    b = np.array([[[1.0], [10.0]], [[2.0], [0.0]]])
    assert do.lora(x, a, b, np.array([1, -1]), np.array([1.0, 0.5]), np.ones((2, 2)))[0].tolist() == [[5, 1], [1, 1]]


# ---------------------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_moe_gb300 as pkg
    return pkg.lib()


BUF, BUF2 = ctypes.c_void_p(256), ctypes.c_void_p(1 << 40)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(257)


def refused(call, good, cases):
    for at, value, rc in cases:
        args = list(good)
        args[at] = value
        assert call(*args) == rc, (at, value)


def test_rows(lib):
    assert lib.moe_w4a16_dispatch_rows(4, 8, 384, 1) == 32
    assert lib.moe_w4a16_dispatch_rows(4, 8, 384, 128) == 32 + 32 * 127
    assert lib.moe_w4a16_dispatch_rows(100, 8, 3, 128) == 800 + 3 * 127
    assert lib.moe_w4a16_dispatch_rows(0, 8, 3, 128) == 0
    for bad in ((-1, 8, 3, 1), (4, 0, 3, 1), (4, 33, 3, 1), (4, 8, 0, 1), (4, 8, 1025, 1), (4, 8, 3, 0),
                (1 << 28, 8, 3, 1), (1 << 20, 8, 1024, 1 << 22)):
        assert lib.moe_w4a16_dispatch_rows(*bad) == -1


ORDER = [(-1, INVALID), (1 << 28, SHAPE)], [(0, INVALID), (33, SHAPE)], [(0, INVALID), (1025, SHAPE)], [(0, INVALID)]


def of_order(M, topk, E, block):
    return [(at, v, rc) for at, cases in zip((M, topk, E, block), ORDER) for v, rc in cases]


def test_sort_refusals(lib):
    good = [BUF, 4, 8, 0, 16, 1, BUF, BUF2, BUF2, None]
    refused(lib.moe_w4a16_dispatch_sort, good, of_order(1, 2, 4, 5) + [
        (0, None, INVALID), (6, None, INVALID), (7, None, INVALID), (8, None, INVALID), (3, -1, INVALID),
        (0, ODD, INVALID), (6, ODD, INVALID), (7, ODD, INVALID), (8, ODD, INVALID)])


def test_gather_refusals(lib):
    good = [BUF, BF16, 64, BUF, BUF, BUF, BUF2, 4, 64, 8, 16, 1, None]
    refused(lib.moe_w4a16_dispatch_gather, good, of_order(7, 9, 10, 11) + [
        (0, None, INVALID), (1, 3, INVALID), (2, 63, INVALID), (3, None, INVALID), (4, None, INVALID), (5, None, INVALID),
        (6, None, INVALID), (8, 0, INVALID), (8, 1 << 23, SHAPE), (0, ODD, INVALID), (6, ODD, INVALID), (3, ODD, INVALID),
        (7, 0, OK)])
    good = [BUF, BF16, 64, BUF, 4, 64, 8, 0, 16, 1, BUF, BUF2, BUF2, BUF2, None]
    refused(lib.moe_w4a16_dispatch_sort_gather, good, of_order(4, 6, 8, 9) + [
        (0, None, INVALID), (1, -1, INVALID), (2, 63, INVALID), (3, None, INVALID), (5, 0, INVALID), (7, -1, INVALID),
        (10, None, INVALID), (11, None, INVALID), (12, None, INVALID), (13, None, INVALID), (13, ODD, INVALID)])


def test_combine_refusals(lib):
    good = [BUF, BF16, BUF, BUF, None, BUF2, BF16, 4, 64, 8, 32, None]
    refused(lib.moe_w4a16_combine, good, [
        (0, None, INVALID), (1, E4M3, INVALID), (2, ODD, INVALID), (3, None, INVALID), (3, ODD, INVALID), (4, ODD, INVALID),
        (5, None, INVALID), (5, ODD, INVALID), (6, 7, INVALID), (7, -1, INVALID), (8, 0, INVALID), (9, 0, INVALID),
        (10, -1, INVALID), (8, 1 << 23, SHAPE), (9, 33, SHAPE), (7, 1 << 28, SHAPE), (7, 0, OK)])
    good = [BUF, BF16, BUF, BF16, BUF, BUF, BUF, BUF, BUF2, BUF2, 4, 64, 8, 16, 1, None]
    refused(lib.moe_w4a16_combine_backward, good, of_order(10, 12, 13, 14) + [
        (at, None, INVALID) for at in (0, 2, 4, 5, 6, 7, 8, 9)] + [(at, ODD, INVALID) for at in (0, 2, 4, 5, 6, 7, 8, 9)] + [
        (1, E4M3, INVALID), (3, E4M3, INVALID), (8, BUF, INVALID), (11, 0, INVALID), (11, 1 << 23, SHAPE), (10, 0, OK)])


def test_route_backward_refusals(lib):
    good = [BUF, BUF, F32, 64, BUF, 4, 64, 8, 1, 1, 1.0, BUF2, None]
    refused(lib.moe_w4a16_route_scored_backward, good, [
        (at, None, INVALID) for at in (0, 1, 4, 11)] + [(at, ODD, INVALID) for at in (0, 1, 4, 11)] + [
        (2, E4M3, INVALID), (3, 63, INVALID), (5, -1, INVALID), (6, 0, INVALID), (6, 1025, SHAPE), (7, 0, INVALID),
        (7, 33, SHAPE), (8, 2, INVALID), (11, BUF, INVALID), (5, (1 << 30) + 1, SHAPE), (5, 0, OK)])


def test_lora_refusals(lib):
    size = lib.moe_w4a16_lora_workspace_size
    assert size(-1, 64, 64, 8, 3) == 0 and size(4, 64, 64, 129, 3) == 0 and size(4, 64, 64, 8, 1024) == 0
    good = [BUF, 64, BUF, BUF, None, BUF, None, F32, BUF2, BF16, 4, 64, 64, 8, 3, BUF, 1 << 40, None]
    refused(lib.moe_w4a16_lora, good, [
        (at, None, INVALID) for at in (0, 2, 3, 5, 8)] + [(at, ODD, INVALID) for at in (0, 2, 3, 4, 5, 6, 8)] + [
        (1, 63, INVALID), (9, E4M3, INVALID), (10, -1, INVALID), (10, (1 << 29) + 1, SHAPE), (11, 0, INVALID),
        (11, 1 << 23, SHAPE), (12, 0, INVALID), (12, 1 << 23, SHAPE), (13, 0, INVALID), (13, 129, SHAPE), (14, 0, INVALID),
        (14, 1024, SHAPE), (15, ctypes.c_void_p(272), INVALID), (6, BUF2, INVALID), (10, 0, OK)])
    need = size(5000, 512, 512, 16, 4)
    if need:
        args = list(good)
        args[1], args[10], args[11], args[12], args[13], args[14], args[16] = 512, 5000, 512, 512, 16, 4, need - 1
        assert lib.moe_w4a16_lora(*args) == WORKSPACE


def test_shared_memory_is_refused(lib):
    """An output that lies in an input, at its first byte, its last, or behind its gaps."""
    at = lambda a: ctypes.c_void_p(a)  # noqa: E731
    base, far = 1 << 20, 1 << 40
    n = 2 * 64 * 4  # of 4 rows of 64 bf16, 4 of them behind a gap of 64: span 7 * 64 * 2
    cases = []
    for out in (base, base + 7 * 128 - 2, base - 32 * 128 + 2):  # (32 rows of an order)
        cases.append((lib.moe_w4a16_dispatch_gather,
                      [at(base), BF16, 128, BUF, BUF, BUF, at(out), 4, 64, 8, 16, 1, None]))
        cases.append((lib.moe_w4a16_dispatch_sort_gather,
                      [at(base), BF16, 128, BUF, 4, 64, 8, 0, 16, 1, BUF, at(far), at(2 * far), at(out), None]))
    for out in (base, base + 32 * 128 - 2, base - n + 2):
        cases.append((lib.moe_w4a16_combine, [at(base), BF16, BUF, BUF, None, at(out), BF16, 4, 64, 8, 32, None]))
    for out in (base + 2, base + n - 2, base - n + 2):
        cases.append((lib.moe_w4a16_combine, [at(far), BF16, BUF, BUF, at(base), at(out), BF16, 4, 64, 8, 32, None]))
        cases.append((lib.moe_w4a16_lora,
                      [at(far), 64, BUF, BUF, None, BUF, at(base), BF16, at(out), BF16, 4, 64, 64, 8, 3, None, 0, None]))
    for out in (base, base + 7 * 128 - 2, base - n + 2):
        cases.append((lib.moe_w4a16_lora,
                      [at(base), 128, BUF, BUF, None, BUF, None, BF16, at(out), BF16, 4, 64, 64, 8, 3, None, 0, None]))
        cases.append((lib.moe_w4a16_route_scored_backward,
                      [BUF, at(base), BF16, 128, BUF, 4, 64, 8, 1, 1, 1.0, at(out), None]))
    for grad, y, w, dy, dw in ((base, far, BUF.value, base, 2 * far), (base, far, BUF.value, base + n - 2, 2 * far),
                               (far, base, BUF.value, base - 32 * 128 + 2, 2 * far), (far, base, BUF.value, base, 2 * far),
                               (far, 2 * far, base, base, base), (far, 2 * far, base, 3 * far, base + 4 * 32 - 4)):
        cases.append((lib.moe_w4a16_combine_backward,
                      [at(grad), BF16, at(y), BF16, at(w), BUF, BUF, BUF, at(dy), at(dw), 4, 64, 8, 16, 1, None]))
    for slots, position in ((far, base), (base, far), (far, base + 4 * 31), (base - 4 * 31, far)):
        cases.append((lib.moe_w4a16_dispatch_sort, [at(base), 4, 8, 0, 16, 1, BUF, at(slots), at(position), None]))
        cases.append((lib.moe_w4a16_dispatch_sort_gather,
                      [at(4 * far), BF16, 64, at(base), 4, 64, 8, 0, 16, 1, BUF, at(slots), at(position), at(2 * far), None]))
    for call, args in cases:
        assert call(*args) == INVALID, (call.__name__, args)
