"""The scored router on the GPU against its float64 definition.

Weights: fp32 arithmetic of a few operations. The argument of the exponential is rounded
to 2^-24 of at most 2^5 (2e-6 of the result), the exponential to 2 ulp, the sums and
quotients to a few more: together below 1e-5 of the result. Rows whose selection hangs
on less than 4e-6 of the scores and values that it compares are left out of the
comparison of ids (equal values are kept in)."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import MoeW4A16Error, routing
from oracle import ops_oracle as oo
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

TOL_W = 1e-5
MARGIN = 4e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def check(logits_t, topk, min_decided=0.95, **kw):
    """Route on the GPU and compare with the oracle on the values that the GPU was given."""
    bias = kw.get("bias")
    ids, w = routing.route_scored(logits_t, topk, **{**kw, "bias": None if bias is None else dev(bias)})
    ref_kw = {**kw, "group_top": kw.get("group_top") or (2 if bias is not None else 1)}
    rid, rw, margin = oo.route_scored(logits_t.float().cpu().numpy(), topk, **ref_kw)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    ok = margin > MARGIN
    assert ok.mean() >= min_decided
    np.testing.assert_array_equal(ids[ok], rid[ok])
    np.testing.assert_allclose(w[ok], rw[ok], rtol=TOL_W, atol=1e-30)
    return ids, w


def normal(M, E, seed, dtype=torch.float32, scale=1.5):
    rng = np.random.default_rng(seed)
    return dev((rng.standard_normal((M, E)) * scale).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("M", [1, 2, 7, 33, 1025])
@pytest.mark.parametrize("E,topk,n_group,topk_group", [
    (384, 8, 1, 1), (256, 8, 8, 4), (160, 6, 8, 3), (64, 6, 1, 1), (1024, 32, 32, 7), (1024, 8, 16, 5),
    (1, 1, 1, 1), (2, 2, 2, 2), (31, 5, 1, 1), (33, 33 % 32, 11, 3), (102, 9, 17, 9), (1020, 12, 17, 3), (6, 3, 3, 2),
    (1000, 20, 1, 1), (48, 4, 16, 4), (320, 1, 5, 1),
])
def test_matches_definition(M, E, topk, n_group, topk_group):
    rng = np.random.default_rng(E + M)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    for scoring, b in (("sigmoid", bias), ("sigmoid", None), ("softmax", bias), ("softmax", None)):
        for dtype in (torch.float32, torch.bfloat16):
            check(normal(M, E, 3 * E + M, dtype), topk, min_decided=0.9 if M > 8 else 0.0, scoring=scoring, bias=b,
                  n_group=n_group, topk_group=topk_group, renormalize=scoring == "sigmoid", scale=2.5)


@pytest.mark.parametrize("group_top", [1, 2])
def test_group_value(group_top):
    # a group with one large value against one with two middling ones
    l = np.full((1, 8), -6.0, np.float32)
    l[0, 1] = 2.0
    l[0, 4:6] = 1.0
    ids, _ = check(dev(l), 1, scoring="sigmoid", n_group=2, topk_group=1, group_top=group_top)
    assert ids[0, 0] == (1 if group_top == 1 else 4)


def test_equal_values_take_the_lowest_ids():
    for E, g, tg in ((384, 1, 1), (256, 8, 4), (99, 3, 2)):
        l = np.round(np.random.default_rng(E).standard_normal((64, E)) * 2).astype(np.float32)  # a handful of values
        check(dev(l), 8, scoring="sigmoid", n_group=g, topk_group=tg, group_top=2)
        check(dev(l), 8, scoring="softmax", n_group=g, topk_group=tg)
        ids, w = check(torch.zeros(3, E, device="cuda"), 8, scoring="softmax", n_group=g, topk_group=tg)
        np.testing.assert_array_equal(ids, np.broadcast_to(np.arange(8), (3, 8)))
        np.testing.assert_allclose(w, 0.125, rtol=TOL_W)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups", [(1, 1), (4, 2)])
def test_masked_logits(scoring, groups):
    rng = np.random.default_rng(7)
    l = rng.standard_normal((12, 64)).astype(np.float32)
    l[0] = -np.inf                                 # nothing to choose
    l[1] = np.nan
    l[2, 5:] = -np.inf                             # fewer than topk left
    l[3, 1::2] = np.nan
    l[4, :60] = -np.inf
    l[5, 10] = np.inf
    l[6, 10] = l[6, 50] = np.inf                   # two that share everything
    l[7] = np.finfo(np.float32).min                # the lowest number is a logit like others
    l[8, ::3] = np.finfo(np.float32).min
    l[9, 16:48] = -np.inf                          # whole groups
    l[10] = np.finfo(np.float32).max
    bias = np.full(64, -0.25, np.float32)          # scores may fall below 0, masked ones stay behind them
    for b in (None, bias):
        for dtype in (torch.float32, torch.bfloat16):
            ids, w = check(dev(l).to(dtype), 8, min_decided=0.7, scoring=scoring, bias=b, n_group=groups[0],
                           topk_group=groups[1])
            assert np.isfinite(w).all()
            assert (w[0] == 0).all() and (w[1] == 0).all()
            assert sorted(set(ids[0])) == sorted(ids[0])


def test_strided_rows_unaligned_rows_and_out():
    big = normal(40, 200, 5)
    for part in (big[:, 3:131], big[:, 4:132], big[::2, :128], big[5:6, 1:129]):
        check(part, 6, min_decided=0.8, scoring="sigmoid", n_group=4, topk_group=2)
        check(part.to(torch.bfloat16)[:, 1:], 6, min_decided=0.8, scoring="softmax")
    ids = torch.full((40, 4), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros((40, 4), dtype=torch.float32, device="cuda")
    got = routing.route_scored(big, 4, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w and (ids >= 0).all()
    assert routing.route_scored(big[:0], 4)[0].shape == (0, 4)


def test_rows_beyond_32_bit_offsets():
    M, E = 2_200_000, 1000  # 2.2e9 logits
    l = torch.zeros(M, E, dtype=torch.bfloat16, device="cuda")
    tail = normal(5, E, 9, torch.bfloat16)
    l[-5:] = tail
    ids, w = routing.route_scored(l, 8, scoring="softmax")
    want = routing.route_scored(tail.contiguous(), 8, scoring="softmax")
    assert torch.equal(ids[-5:], want[0]) and torch.equal(w[-5:], want[1])


def test_other_stream_and_repeat():
    l = normal(513, 384, 11)
    a = routing.route_scored(l, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = routing.route_scored(l, 8, stream=s)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_ids_and_weights_feed_the_forward():
    from int4_weight_only_moe_gb300 import inputs
    from tests.gpu_helpers import Problem, assert_close, bf16_tensor_to_f64, bits16
    p = Problem(16, 256, 128, 4)
    hidden = inputs.hidden_states(9, 256)
    ids, w = routing.route_scored(normal(9, 16, 2), 4, bias=dev(np.linspace(-0.1, 0.1, 16).astype(np.float32)),
                                  n_group=4, topk_group=2, scale=2.5)
    out = bf16_tensor_to_f64(p.moe.forward(dev(bits16(hidden)), ids, w))
    assert_close(out, p.reference(hidden, ids.cpu().numpy(), w.cpu().numpy()), "scored routing")
    p.close()


def test_refusals():
    l = normal(4, 64, 1)
    with pytest.raises(MoeW4A16Error):
        routing.route_scored(l, 8, n_group=5)
    with pytest.raises(MoeW4A16Error):
        routing.route_scored(l, 33)
    with pytest.raises(ValueError):
        routing.route_scored(l, 8, scoring="tanh")
    with pytest.raises(ValueError):
        routing.route_scored(l, 8, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(ValueError):
        routing.route_scored(l.t(), 2)
    with pytest.raises(ValueError):
        routing.route_scored(l, 8, ids=torch.zeros(4, 7, dtype=torch.int32, device="cuda"))
