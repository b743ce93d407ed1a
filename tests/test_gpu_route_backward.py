"""Gradient of the scored router's weights on the GPU against its 64-bit formula and against
differences of the 64-bit weights.

Tolerances, in units of 2^-24 of the size of a gradient's terms: the exponentials are within
2 ulp of their argument's, whose difference to the row's largest is rounded once (|x| units
more, at most 60 here, for a softmax), sums of up to E / 32 + 5 terms one after another,
quotients and products below 20 in all."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import MoeW4A16Error, routing
from oracle import dispatch_oracle as do
from tests.gpu_helpers import dev

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
UNITS = 20 + 32 + 5 + 60
SMALL = 2.0 ** -126  # below this fp32 has no full precision


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def check(l, ids, scoring, renormalize, scale=2.5, seed=0, **kw):
    g = np.random.default_rng(seed).standard_normal(ids.shape).astype(np.float32)
    got = routing.route_scored_backward(dev(g), l, dev(ids), scoring=scoring, renormalize=renormalize, scale=scale, **kw)
    assert got.dtype == l.dtype
    want, size = do.route_backward(g, l.float().cpu().numpy(), ids, scoring, renormalize, scale)
    out = got.float().cpu().numpy().astype(np.float64)
    over = np.abs(out - want) - HALF[l.dtype] * np.abs(want) - UNITS * 2.0 ** -24 * size - SMALL
    assert (over <= 0).all(), over.max()
    return got


def logits(M, E, seed, dtype, by=1.5):
    return dev((np.random.default_rng(seed).standard_normal((M, E)) * by).astype(np.float32)).to(dtype)


def chosen(l, topk, seed):
    """Ids such as a biased selection gives: mostly the best, not always."""
    noise = np.random.default_rng(seed).standard_normal(tuple(l.shape))
    return np.argsort(-(l.float().cpu().numpy() + noise), 1)[:, :topk].astype(np.int32)


@pytest.mark.parametrize("M", [1, 3, 130])
@pytest.mark.parametrize("E,topk", [(384, 8), (256, 8), (160, 6), (1, 1), (31, 5), (33, 32), (1024, 32), (1001, 1), (8, 8)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_matches_the_formula(M, E, topk, scoring, renormalize):
    for dtype in (torch.float32, torch.bfloat16):
        l = logits(M, E, E + M, dtype)
        check(l, chosen(l, topk, M), scoring, renormalize)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_against_differences(scoring, renormalize):
    # of the 64-bit weights, with a step of 1e-5: their own error is below 1e-9 of the values
    l, scale = logits(6, 40, 1, torch.float32), 2.5
    ids = chosen(l, 5, 2)
    g = np.random.default_rng(0).standard_normal(ids.shape).astype(np.float32)
    got = check(l, ids, scoring, renormalize, scale).cpu().numpy()
    x = l.cpu().numpy().astype(np.float64)
    loss = lambda v: (do.route_weights(v, ids, scoring, renormalize, scale) * g).sum(1)  # noqa: E731
    for e in range(40):
        d = np.zeros_like(x)
        d[:, e] = 1e-5
        np.testing.assert_allclose(got[:, e], (loss(x + d) - loss(x - d)) / 2e-5, atol=3e-6)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_edges(scoring, renormalize):
    l = np.random.default_rng(3).standard_normal((12, 64)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2, 5:] = -np.inf
    l[3, 1::2] = np.nan
    l[4, 10] = np.inf
    l[5, 10] = l[5, 20] = np.inf
    l[6] = np.finfo(np.float32).min
    l[7] = 80.0
    l[8] = -80.0
    l[9, ::2] = -50.0
    ids = np.stack([np.random.default_rng(t).permutation(64)[:8] for t in range(12)]).astype(np.int32)
    ids[4, 0] = ids[5, 0] = 10
    ids[5, 1] = 20
    ids[10] = [3, 3, 3, 7, -1, 64, 7, 9]       # the same expert twice and three times, no expert
    ids[11] = -1
    for dtype in (torch.float32, torch.bfloat16):
        got = check(dev(l).to(dtype), ids, scoring, renormalize)
        assert torch.isfinite(got).all()
        assert not got[0].any() and not got[1].any() and not got[11].any()


def test_strided_logits_out_stream_and_graph():
    big = logits(40, 200, 5, torch.float32)
    for l in (big[:, 3:131], big[::2, :128], big[5:6, 1:129]):
        ids = chosen(l, 6, 1)
        want = check(l, ids, "sigmoid", True)
        out = torch.empty(l.shape, device="cuda")
        assert torch.equal(check(l, ids, "sigmoid", True, out=out), want)
    l, ids = logits(300, 384, 6, torch.float32), None
    ids = dev(chosen(l, 8, 1))
    g = torch.randn(300, 8, device="cuda")
    first = routing.route_scored_backward(g, l, ids)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = routing.route_scored_backward(g, l, ids, stream=s)
    s.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = routing.route_scored_backward(g, l, ids)
    g.mul_(2.0)
    graph.replay()
    assert torch.equal(kept, first * 2.0)  # (a power of two goes through every product)
    assert routing.route_scored_backward(g[:0], l[:0], ids[:0]).shape == (0, 384)


def test_behind_the_router():
    l = logits(64, 96, 8, torch.float32)
    bias = dev(np.random.default_rng(1).standard_normal(96).astype(np.float32) * 0.1)
    ids, w = routing.route_scored(l, 6, bias=bias, n_group=8, topk_group=4, scale=2.5)
    check(l, ids.cpu().numpy(), "sigmoid", True)


def test_refusals():
    l = logits(4, 64, 1, torch.float32)
    ids, g = torch.zeros(4, 8, dtype=torch.int32, device="cuda"), torch.zeros(4, 8, device="cuda")
    with pytest.raises(MoeW4A16Error):
        routing.route_scored_backward(g, l, ids, out=l)
    for call in (lambda: routing.route_scored_backward(g, l, ids.long()), lambda: routing.route_scored_backward(g[:3], l, ids),
                 lambda: routing.route_scored_backward(g, l, ids, scoring="tanh"),
                 lambda: routing.route_scored_backward(g, l.t(), ids), lambda: routing.route_scored_backward(g, l, ids[0]),
                 lambda: routing.route_scored_backward(g.double(), l, ids),
                 lambda: routing.route_scored_backward(g, l, ids, out=torch.zeros(4, 63, device="cuda"))):
        with pytest.raises(ValueError):
            call()
