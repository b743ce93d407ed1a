"""The operators around the routed experts, without a GPU: the oracle's definitions on
values known by hand, and the refusals of the C entry points and of the Python calls."""
import ctypes

import numpy as np
import pytest

from oracle import ops_oracle as oo

OK, INVALID, SHAPE, WORKSPACE = 0, -1, -2, -3
F32, BF16 = 0, 1


# ---------------------------------------------------------------------- the definitions


@pytest.mark.parametrize("byte,value", [(0x00, 0.0), (0x01, 2.0 ** -9), (0x07, 7 * 2.0 ** -9), (0x08, 2.0 ** -6),
                                        (0x38, 1.0), (0x39, 1.125), (0xB8, -1.0), (0x7E, 448.0), (0xFE, -448.0)])
def test_e4m3_values(byte, value):
    assert oo.e4m3_values([byte])[0] == value


def test_e4m3_not_a_number():
    assert np.isnan(oo.e4m3_values([0x7F, 0xFF])).all()


@pytest.mark.parametrize("v,want", [(1.0625, 1.0), (1.1875, 1.25), (1.07, 1.125), (-1.0625, -1.0), (500.0, 448.0),
                                    (2.0 ** -10, 0.0), (3 * 2.0 ** -10, 2.0 ** -8), (447.9, 448.0), (0.0, 0.0)])
def test_e4m3_rounds_to_nearest_even(v, want):
    assert oo.e4m3_round(v) == want


def test_quantize_by_hand():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 1], x[0, 129] = 896.0, -3.0, 7.0
    q, s = oo.quantize(x)
    assert s[0, 0] == 2.0 and q[0, 0] == 448.0 and q[0, 1] == -1.5
    assert s[0, 1] == np.float32(7.0 / 448.0) and q[0, 129] == 448.0
    assert s[1, 0] == np.float32(2.0 ** -126) and not q[1].any()


def test_route_by_hand():
    # two groups of two: the biased choice takes group 1, the weights are unbiased
    l = np.array([[2.0, 1.0, 0.0, 0.5]])
    bias = np.array([0.0, 0.0, 1.0, 1.0])
    ids, w, _ = oo.route_scored(l, 2, "sigmoid", bias, 2, 1, 2)
    assert ids.tolist() == [[3, 2]]
    s3, s2 = 1 / (1 + np.exp(-0.5)), 0.5
    np.testing.assert_allclose(w, [[s3 / (s3 + s2), s2 / (s3 + s2)]])
    # equal logits: lowest id first; masked ones last, with weight 0
    ids, w, _ = oo.route_scored(np.array([[1.0, 1.0, -np.inf, np.nan]]), 3, "softmax")
    assert ids.tolist() == [[0, 1, 2]] and w.tolist() == [[0.5, 0.5, 0.0]]
    ids, w, _ = oo.route_scored(np.full((1, 4), -np.inf), 2, "softmax")
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


# -------------------------------------------------------------------------- refusals


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import int4_weight_only_moe_gb300 as pkg
    return pkg.lib()


BUF = ctypes.c_void_p(256)  # never dereferenced: validation fails first


def _route(lib, logits=BUF, kind=F32, stride=64, M=4, E=64, topk=4, scoring=1, bias=None, n_group=4, topk_group=2,
           group_top=2, ids=BUF, w=BUF):
    return lib.moe_w4a16_route_scored(logits, kind, stride, M, E, topk, scoring, bias, n_group, topk_group, group_top,
                                      1, 1.0, ids, w, None)


@pytest.mark.parametrize("change,rc", [
    (dict(kind=2), INVALID), (dict(scoring=2), INVALID), (dict(M=-1), INVALID), (dict(E=0), INVALID),
    (dict(topk=0), INVALID), (dict(E=2048, n_group=1, topk_group=1, stride=2048), SHAPE),
    (dict(topk=33, E=256, stride=256), SHAPE), (dict(n_group=0), INVALID), (dict(n_group=3), INVALID),
    (dict(n_group=64, topk_group=32), SHAPE), (dict(topk_group=0), INVALID), (dict(topk_group=5), INVALID),
    (dict(group_top=0), INVALID), (dict(group_top=3), INVALID), (dict(topk=32, topk_group=1), INVALID),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(stride=63), INVALID),
    (dict(logits=ctypes.c_void_p(258)), INVALID), (dict(bias=ctypes.c_void_p(257)), INVALID),
    (dict(M=0, logits=None, ids=None, w=None), OK),
])
def test_route_scored_refusals(lib, change, rc):
    assert _route(lib, **change) == rc
    if rc != OK:
        assert lib.moe_w4a16_last_error()


@pytest.mark.parametrize("name", ["moe_w4a16_fp8_quantize", "moe_w4a16_fp8_swiglu_quantize",
                                  "moe_w4a16_fp8_quantize_weight"])
def test_quantize_refusals(lib, name):
    call = getattr(lib, name)
    width = 512 if "swiglu" in name else 256
    good = [BUF, F32, width, 4, 256, BUF, BUF, None]
    for at, value, rc in [(0, None, INVALID), (1, 7, INVALID), (2, width - 1, INVALID), (3, -1, INVALID),
                          (4, 0, INVALID), (4, 1 << 23, SHAPE), (5, None, INVALID), (6, None, INVALID),
                          (0, ctypes.c_void_p(257), INVALID), (6, ctypes.c_void_p(258), INVALID), (3, 0, OK)]:
        args = list(good)
        args[at] = value
        assert call(*args) == rc, (at, value)


def test_matmul_refusals(lib):
    good = [BUF, 256, BUF, BUF, 256, BUF, None, BUF, F32, 4, 128, 256, None]
    for at, value, rc in [(0, None, INVALID), (2, None, INVALID), (3, None, INVALID), (5, None, INVALID),
                          (7, None, INVALID), (1, 255, INVALID), (4, 255, INVALID), (8, 5, INVALID),
                          (9, -1, INVALID), (10, -1, INVALID), (11, 0, INVALID), (10, 1 << 23, SHAPE),
                          (11, 1 << 23, SHAPE), (2, ctypes.c_void_p(258), INVALID), (6, ctypes.c_void_p(257), INVALID),
                          (7, ctypes.c_void_p(258), INVALID), (9, 0, OK), (10, 0, OK)]:
        args = list(good)
        args[at] = value
        assert lib.moe_w4a16_fp8_matmul(*args) == rc, (at, value)


def test_shared_expert_refusals(lib):
    size = lib.moe_w4a16_shared_expert_workspace_size
    need = size(4, 256, 128)
    assert need > 0 and size(8, 256, 128) >= need
    assert size(-1, 256, 128) == 0 and size(4, 200, 128) == 0 and size(4, 256, 96) == 0
    good = [BUF, BUF, BUF, BUF, BUF, None, BUF, 4, 256, 128, BUF, need, None]
    for at, value, rc in [(i, None, INVALID) for i in (0, 1, 2, 3, 4, 6)] + [
            (7, -1, SHAPE), (8, 200, SHAPE), (9, 96, SHAPE), (8, 0, SHAPE), (11, need - 1, WORKSPACE),
            (10, ctypes.c_void_p(272), INVALID), (2, ctypes.c_void_p(258), INVALID), (7, 0, OK)]:
        args = list(good)
        args[at] = value
        assert lib.moe_w4a16_shared_expert(*args) == rc, (at, value)


def test_set_option_refusals(lib):
    for option, value, rc in [(0, 0, INVALID), (3, 1, INVALID), (1, -1, INVALID), (2, 2, INVALID), (1, 0, OK), (2, 0, OK)]:
        assert lib.moe_w4a16_fp8_set_option(option, value) == rc


def test_python_calls_refuse_host_tensors_and_shapes():
    import torch
    from int4_weight_only_moe_gb300 import fp8, routing
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="CUDA"):
        routing.route_scored(x, 2)
    with pytest.raises(ValueError, match="two dimensions"):
        routing.route_scored(x[0], 2)
    with pytest.raises(ValueError, match="dtype"):
        routing.route_scored(x.double(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.quantize(x)
    with pytest.raises(ValueError, match="even"):
        fp8.swiglu_quantize(torch.zeros(4, 255))
    with pytest.raises(ValueError, match="dtype"):
        fp8.matmul(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.matmul(x.to(torch.uint8), x, x.to(torch.uint8), x)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.shared_expert(x.bfloat16(), x.to(torch.uint8), x, torch.zeros(128, 128, dtype=torch.uint8), x)
