"""Every output of the order, gather, combine, gradients and adapters against every input that
the same launch reads: a call in which they share a byte is refused, one in which they only
touch is not. The host code on the fake CUDA runtime, so that nothing is launched."""
import ctypes

import pytest

from tests.test_host_code_dispatch_cpu import BF16, F32, lib, library  # noqa: F401 (fixtures)

INVALID = -1
M, K, TOPK, E, BLOCK = 5, 64, 3, 7, 4
ROWS = M * TOPK + E * (BLOCK - 1)
IDS, OFFSETS, SLOTS = 4 * M * TOPK, 4 * (E + 1), 4 * ROWS
R, N, L = 8, 48, 3

# arguments by name (in the call's order), then the bytes of the arrays: inputs, outputs
CALLS = {
    "moe_w4a16_dispatch_sort": ([("ids", "p"), M, TOPK, 0, E, BLOCK, ("offsets", "p"), ("slots", "p"), ("position", "p"), None],
                                dict(ids=IDS), dict(offsets=OFFSETS, slots=SLOTS, position=IDS)),
    "moe_w4a16_dispatch_gather": ([("x", "p"), BF16, K, ("offsets", "p"), ("slots", "p"), ("position", "p"), ("out", "p"), M, K, TOPK, E,
                                   BLOCK, None],
                                  dict(x=2 * M * K, offsets=OFFSETS, slots=SLOTS, position=IDS), dict(out=2 * ROWS * K)),
    "moe_w4a16_dispatch_sort_gather": ([("x", "p"), BF16, K, ("ids", "p"), M, K, TOPK, 0, E, BLOCK, ("offsets", "p"), ("slots", "p"),
                                        ("position", "p"), ("out", "p"), None],
                                       dict(x=2 * M * K, ids=IDS), dict(offsets=OFFSETS, slots=SLOTS, position=IDS, out=2 * ROWS * K)),
    "moe_w4a16_combine": ([("y", "p"), BF16, ("w", "p"), ("position", "p"), ("add", "p"), ("out", "p"), F32, M, K, TOPK, ROWS, None],
                          dict(y=2 * ROWS * K, w=IDS, position=IDS, add=4 * M * K), dict(out=4 * M * K)),
    "moe_w4a16_combine_backward": ([("g", "p"), F32, ("y", "p"), BF16, ("w", "p"), ("offsets", "p"), ("slots", "p"), ("position", "p"),
                                    ("dy", "p"), ("dw", "p"), M, K, TOPK, E, BLOCK, None],
                                   dict(g=4 * M * K, y=2 * ROWS * K, w=IDS, offsets=OFFSETS, slots=SLOTS, position=IDS),
                                   dict(dy=2 * ROWS * K, dw=IDS)),
    "moe_w4a16_route_scored_backward": ([("dw", "p"), ("l", "p"), F32, E, ("ids", "p"), M, E, TOPK, 1, 1, 1.0, ("dl", "p"), None],
                                        dict(dw=IDS, l=4 * M * E, ids=IDS), dict(dl=4 * M * E)),
    "moe_w4a16_lora": ([("x", "p"), K, ("a", "p"), ("b", "p"), ("scale", "p"), ("index", "p"), ("add", "p"), BF16, ("out", "p"), F32, M, K,
                        N, R, L, None, 0, None],
                       dict(x=2 * M * K, a=2 * L * R * K, b=2 * L * N * R, scale=4 * L, index=4 * M, add=2 * M * N), dict(out=4 * M * N)),
}
PAIRS = [(call, i, o) for call, (_, ins, outs) in CALLS.items() for i in ins for o in outs]


def addresses(names):
    return {name: (i + 1) << 32 for i, name in enumerate(names)}


def call(lib, name, at):  # noqa: F811
    args = [ctypes.c_void_p(at[a[0]]) if isinstance(a, tuple) else a for a in CALLS[name][0]]
    return getattr(lib, name)(*args)


@pytest.mark.parametrize("name,i,o", PAIRS)
def test_outputs_in_inputs(lib, name, i, o):  # noqa: F811
    _, ins, outs = CALLS[name]
    at = addresses([*ins, *outs])
    assert call(lib, name, at) == 0
    a = at[i]
    for where in (a, a + ins[i] - 4, a - outs[o] + 4):
        before = lib.fake_launches()
        if i == "add" and where == a and name == "moe_w4a16_combine":  # (in place)
            assert call(lib, name, {**at, o: where}) == 0
            continue
        assert call(lib, name, {**at, o: where}) == INVALID, hex(where - a)
        assert lib.fake_launches() == before
    for where in (a + ins[i], a - outs[o]):
        assert call(lib, name, {**at, o: where}) == 0


def test_rows_far_apart_leave_room_between_them(lib):  # noqa: F811
    """An output between two rows of a strided input shares no byte with it."""
    base, far = 1 << 32, 1 << 40
    p = ctypes.c_void_p
    stride = 1 << 20  # elements

    def lora(out, m=M):
        return lib.moe_w4a16_lora(p(base), stride, p(far), p(2 * far), None, p(3 * far), None, F32, p(out), F32, m, K, N, R, L, None, 0,
                                  None)

    for row in range(M - 1):
        first, end = base + 2 * row * stride + 2 * K, base + 2 * (row + 1) * stride
        assert lora(first) == 0 and lora(end - 4 * M * N) == 0
        assert lora(first - 4) == INVALID and lora(end - 4 * M * N + 4) == INVALID
    assert lora(base + 2 * (M - 1) * stride + 2 * K) == 0 and lora(base + 2 * (M - 1) * stride + 2 * K - 4) == INVALID
    assert lora(base + 2 * stride, 1) == 0  # (one row: its stride says nothing)
    # as many rows of the output as fill a gap and reach the next row
    for rows, rc in ((M, 0), (4096, INVALID)):
        assert lib.moe_w4a16_route_scored_backward(p(far), p(base), F32, stride, p(2 * far), rows, 256, TOPK, 1, 1, 1.0,
                                                   p(base + 4096), None) == rc
