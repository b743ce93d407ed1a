"""The scored router on rows whose logits lie far apart: without a bias the ids are those that
the logits order (a softmax's scores from 104 below the row's largest logit on are 0 in fp32,
and equal); with one they are those of fp32 scores, down to 2^-149."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import routing
from tests.gpu_helpers import dev
from tests.test_gpu_fp8 import _built  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def ids_by(values, group_values, topk, n_group, topk_group):
    """The topk largest values of each row in its best groups; equal ones: lower index first."""
    M, E = values.shape
    size = E // n_group
    out = np.empty((M, topk), np.int64)
    for t in range(M):
        groups = np.sort(np.argsort(-group_values[t], kind="stable")[:topk_group])
        cand = (groups[:, None] * size + np.arange(size)).reshape(-1)
        out[t] = cand[np.argsort(-values[t, cand], kind="stable")[:topk]]
    return out


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,n_group,topk_group", [(384, 1, 1), (256, 8, 4), (160, 8, 3), (33, 11, 3), (1020, 17, 5)])
def test_without_a_bias_the_logits_decide(scoring, dtype, E, n_group, topk_group):
    rng = np.random.default_rng(E)
    l = dev((rng.standard_normal((300, E)) * 60).astype(np.float32)).to(dtype)
    l[:100, ::7] += 300.0
    l[100:200] = l[100:200].round()  # (equal ones among them)
    l[200:, 1::3] = -0.0
    l[200:, 2::3] = 0.0
    topk = min(8, topk_group * (E // n_group))
    ids, w = routing.route_scored(l, topk, scoring=scoring, n_group=n_group, topk_group=topk_group)
    l64 = l.float().cpu().numpy().astype(np.float64)
    if scoring == "softmax":
        l64 = np.where(l64 < l64.max(1, keepdims=True) - 104, -1e30, l64)
    want = ids_by(l64, l64.reshape(300, n_group, -1).max(2), topk, n_group, topk_group)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    assert w.isfinite().all()


@pytest.mark.parametrize("bias", [None, 0.0], ids=["no bias", "zeros"])
@pytest.mark.parametrize("n_group,topk_group,group_top", [(1, 1, 1), (4, 3, 1), (4, 3, 2), (4, 2, 2)])
def test_softmax_scores_below_the_normal_numbers(bias, n_group, topk_group, group_top):
    # one logit of 0, the others -88 to -100 in steps of 0.4: scores from 6e-39 to 3.7e-44,
    # neighbours a factor of 1.49 apart (at the smallest 27 and 40 units of 2^-149)
    E = 32
    rng = np.random.default_rng(3)
    l = np.empty((50, E), np.float32)
    for t in range(50):
        l[t, rng.permutation(E)] = np.concatenate([[0.0], -88 - 0.4 * np.arange(E - 1)])
    b = None if bias is None else torch.full((E,), bias, device="cuda")
    topk = topk_group * (E // n_group)
    ids, _ = routing.route_scored(dev(l), topk, scoring="softmax", bias=b, n_group=n_group, topk_group=topk_group,
                                  group_top=group_top)
    s = np.exp(l.astype(np.float64))
    best = np.sort(s.reshape(50, n_group, -1), 2)[:, :, ::-1]
    np.testing.assert_array_equal(ids.cpu().numpy(), ids_by(s, best[:, :, :group_top].sum(2), topk, n_group, topk_group))


def test_sigmoid_scores_below_the_normal_numbers():
    # logits of -87.4 to -88.6, scores from 1.1e-38 to 3.3e-39
    l = np.full((1, 8), -88.6, np.float32)
    l[0, 5], l[0, 2] = -87.4, -88.0
    ids, _ = routing.route_scored(dev(l), 3, scoring="sigmoid", bias=torch.zeros(8, device="cuda"))
    assert ids.tolist() == [[5, 2, 0]]


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("far", [1, 5, 20, 40, 60, 70])
def test_scores_further_apart_than_the_stated_error_keep_their_order(scoring, far):
    # neighbours differ by twice the error of a score, 4 x 2^-22 + far 2^-23 of it, and by two
    # ulps of the logits' own rounding (scores of 3e-37 and more: below 2^-126 their own spacing counts)
    E = 32
    step = 2 * (4 * 2.0 ** -22 + far * 2.0 ** -23) + 2 * float(np.spacing(np.float32(far)))
    rng = np.random.default_rng(far)
    l = np.empty((200, E), np.float32)
    for t in range(200):
        l[t, rng.permutation(E)] = np.concatenate([[0.0], -far * (1 + 0.2 * rng.random()) - step * np.arange(E - 1)])
    ids, _ = routing.route_scored(dev(l), E, scoring=scoring, bias=torch.zeros(E, device="cuda"))
    np.testing.assert_array_equal(ids.cpu().numpy(), np.argsort(-l, 1, kind="stable"))
