"""The whole layer with low-rank adapters beside the shared expert, against the definitions of
its parts, within the layer's tolerance (test_gpu_layer.py); rows without an adapter as the
layer without adapters gives them, but for the order of roundings."""
import subprocess
import sys

import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8, inputs
from int4_weight_only_moe_gb300.layer import MoELayer
from oracle import dispatch_oracle as do
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
    E, K, N, k, L, r = 16, 256, 128, 4, 5, 16
    p = Problem(E, K, N, k)
    rng = np.random.default_rng(0)
    w = lambda *s: dev((rng.standard_normal(s) * s[-1] ** -0.5).astype(np.float32))  # noqa: E731
    shared = fp8.quantize_weight(w(2 * N, K)) + fp8.quantize_weight(w(K, N))
    adapters = (w(L, r, K).bfloat16(), w(L, 2 * N, r).bfloat16(), dev(rng.random(L).astype(np.float32) + 0.5))
    yield p, shared, adapters
    p.close()


@pytest.mark.parametrize("M", [1, 3, 33, 150, 1000])
def test_layer(parts, M):
    p, shared, adapters = parts
    layer = MoELayer(p.moe, shared, scale=2.5, adapters=adapters)
    hidden = inputs.hidden_states(M, p.K, step=M)
    x = dev(bits16(hidden)).view(torch.bfloat16)
    index = np.random.default_rng(M).integers(-1, 5, M).astype(np.int32)
    out, ids, w = layer.forward(x, dev(inputs.router_logits(M, p.E, "normal", step=M)), adapter=dev(index))
    routed = p.reference(hidden, ids.cpu().numpy(), w.cpu().numpy())
    w1, w1_s, w2, w2_s = [oo.e4m3_values(t.view(torch.uint8).cpu().numpy()) if i % 2 == 0 else t.cpu().numpy()
                          for i, t in enumerate(shared)]
    h = inputs.bf16_bits_to_f32(hidden).astype(np.float64)
    gu, _ = oo.matmul(*oo.quantize(h), w1, w1_s)
    gu = do.lora(h, *(t.float().cpu().numpy() for t in adapters[:2]), index, adapters[2].cpu().numpy(), gu)[0]
    act = oo.silu(gu[:, :p.N]) * gu[:, p.N:]
    want, _ = oo.matmul(*oo.quantize(act), w2, w2_s, routed)
    rel, _ = errors(bf16_tensor_to_f64(out), want)
    rms = np.sqrt(np.mean(want ** 2))
    over = np.abs(bf16_tensor_to_f64(out) - want) - BF16_HALF_ULP_REL * (np.abs(want) + np.abs(routed))
    assert rel <= TOL_REL_L2 and over.max() / rms <= TOL_MAX_OVER_RMS
    assert p.moe.status() == 0 and fp8.status() == 0


def test_on_another_stream_and_captured(parts):
    p, shared, adapters = parts
    layer = MoELayer(p.moe, shared, adapters=adapters)
    x, l = torch.randn(40, p.K, device="cuda").bfloat16(), torch.randn(40, p.E, device="cuda")
    index = torch.randint(-1, 5, (40,), device="cuda", dtype=torch.int32)
    want = layer.forward(x, l, adapter=index)[0].float()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer.forward(x, l, stream=s, adapter=index)[0]
    s.synchronize()
    # (the routed experts' fp32 sum is taken in no fixed order: half an ulp of bf16 either way)
    assert (got.float() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.forward(x, l, adapter=index)[0]
    graph.replay()
    torch.cuda.synchronize()
    assert (out.float() - want).abs().max() <= 2.0 ** -7 * want.abs().max()


def test_refusals(parts):
    p, shared, adapters = parts
    x, l = torch.zeros(4, p.K, device="cuda", dtype=torch.bfloat16), torch.zeros(4, p.E, device="cuda")
    index = torch.zeros(4, device="cuda", dtype=torch.int32)
    with pytest.raises(ValueError):
        MoELayer(p.moe, None, adapters=adapters)
    with pytest.raises(ValueError):
        MoELayer(p.moe, shared).forward(x, l, adapter=index)
    with pytest.raises(ValueError):
        MoELayer(p.moe, shared, adapters=adapters).forward(x, l, adapter=index[:3])
    with pytest.raises(ValueError):
        MoELayer(p.moe, shared, adapters=(adapters[0], adapters[1][:, :-8].contiguous())).forward(x, l, adapter=index)


def test_example_runs():
    r = subprocess.run([sys.executable, "examples/moe_layer.py", "--tokens", "9", "--experts", "16", "--hidden", "256",
                        "--inter", "128", "--topk", "4", "--adapters", "3"], cwd=ROOT, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr
    assert "status 0 / 0" in r.stdout
