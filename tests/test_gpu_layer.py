"""The whole layer -- scored router, W4A16 routed experts, 8-bit shared expert -- against
the definitions of its parts, from one token on, within the feed-forward's tolerance. The
routed sum is rounded to bf16 before the shared expert adds to it, which the bf16 output's
own rounding covers once more (2^-8 of it)."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8, inputs
from int4_weight_only_moe_gb300.layer import MoELayer
from oracle import ops_oracle as oo
from tests.conftest import ROOT
from tests.gpu_helpers import BF16_HALF_ULP_REL, Problem, TOL_MAX_OVER_RMS, TOL_REL_L2, bf16_tensor_to_f64, bits16, dev, errors

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture(scope="module")
def parts():
    E, K, N, k = 32, 256, 128, 4
    p = Problem(E, K, N, k)
    rng = np.random.default_rng(0)
    w = lambda *s: dev((rng.standard_normal(s) * s[1] ** -0.5).astype(np.float32))
    shared = fp8.quantize_weight(w(2 * N, K)) + fp8.quantize_weight(w(K, N))
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    yield p, shared, bias
    p.close()


@pytest.mark.parametrize("M", [1, 3, 33, 150, 700])
@pytest.mark.parametrize("with_shared", [True, False])
def test_layer(parts, M, with_shared):
    p, shared, bias = parts
    layer = MoELayer(p.moe, shared if with_shared else None, bias=dev(bias), n_group=4, topk_group=2, scale=2.5)
    hidden = inputs.hidden_states(M, p.K, step=M)
    logits = inputs.router_logits(M, p.E, "normal", step=M)
    x = dev(bits16(hidden)).view(torch.bfloat16)
    out, ids, w = layer.forward(x, dev(logits))
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    rid, rw, margin = oo.route_scored(logits, p.topk, "sigmoid", bias, 4, 2, 2, True, 2.5)
    sure = margin > 4e-6
    np.testing.assert_array_equal(ids[sure], rid[sure])
    np.testing.assert_allclose(w[sure], rw[sure], rtol=1e-5)
    routed = p.reference(hidden, ids, w)
    want = routed
    if with_shared:
        q = [oo.e4m3_values(t.view(torch.uint8).cpu().numpy()) if i % 2 == 0 else t.cpu().numpy()
             for i, t in enumerate(shared)]
        want = oo.shared_expert(inputs.bf16_bits_to_f32(hidden).astype(np.float64), *q, add=routed)
    got = bf16_tensor_to_f64(out)
    rel, _ = errors(got, want)
    rms = np.sqrt(np.mean(want ** 2))
    over = np.abs(got - want) - BF16_HALF_ULP_REL * (np.abs(want) + np.abs(routed))
    assert rel <= TOL_REL_L2 and over.max() / rms <= TOL_MAX_OVER_RMS
    assert p.moe.status() == 0 and fp8.status() == 0


def test_layer_on_another_stream(parts):
    p, shared, bias = parts
    layer = MoELayer(p.moe, shared, bias=dev(bias), n_group=4, topk_group=2)
    x = torch.randn(40, p.K, device="cuda").bfloat16()
    l = torch.randn(40, p.E, device="cuda")
    want = layer.forward(x, l)[0].float()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer.forward(x, l, stream=s)[0]
    s.synchronize()
    # (the routed experts' fp32 sum is taken in no fixed order: it may round to the other
    # neighbour, half an ulp of bf16 either way)
    assert (got.float() - want).abs().max() <= 2.0 ** -7 * want.abs().max()


def test_layer_refusals(parts):
    p, shared, _ = parts
    layer = MoELayer(p.moe, shared)
    x = torch.zeros(4, p.K, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layer.forward(x, torch.zeros(4, p.E + 1, device="cuda"))
    with pytest.raises(ValueError):
        layer.forward(x, torch.zeros(3, p.E, device="cuda"))


def test_example_runs():
    r = subprocess.run([sys.executable, "examples/moe_layer.py", "--tokens", "9", "--experts", "16", "--hidden", "256",
                        "--inter", "128", "--topk", "4"], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr
    assert "status 0 / 0" in r.stdout
