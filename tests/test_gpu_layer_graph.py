"""The whole layer in a CUDA graph, and with no tokens."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8
from int4_weight_only_moe_gb300.layer import MoELayer
from tests.gpu_helpers import Problem, dev
from tests.test_gpu_fp8 import _built, expert, rand  # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def layer():
    p = Problem(32, 256, 128, 4)
    yield MoELayer(p.moe, expert(256, 128, 6), bias=dev(np.linspace(-0.1, 0.1, 32).astype(np.float32)), n_group=4,
                   topk_group=2, scale=2.5)
    p.close()


@pytest.mark.parametrize("M", [1, 3, 40, 150])
def test_layer_replays_from_a_cuda_graph(layer, M):
    x, logits = rand((M, 256), 1), rand((M, 32), 2, dtype=torch.float32)
    layer.forward(x, logits)  # (the routed experts' workspace is made outside the capture)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, ids, w = layer.forward(x, logits)
    for seed in (3, 4, 5):
        x.copy_(rand((M, 256), seed))
        logits.copy_(rand((M, 32), seed + 10, dtype=torch.float32))
        g.replay()
        torch.cuda.synchronize()
        want = layer.forward(x, logits)
        assert torch.equal(ids, want[1]) and torch.equal(w, want[2])
        # (the routed experts' fp32 sums are taken in no fixed order: half an ulp of bf16 either way)
        assert (out - want[0]).abs().float().max() <= 2.0 ** -7 * want[0].abs().float().max()
    assert fp8.status() == 0 and layer.experts.status() == 0


def test_layer_of_no_tokens(layer):
    out, ids, w = layer.forward(rand((1, 256), 1)[:0], torch.zeros(0, 32, device="cuda"))
    assert out.shape == (0, 256) and ids.shape == (0, 4) and w.shape == (0, 4)
