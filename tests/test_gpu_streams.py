"""Calls on a stream other than the current one, while work queued on the current stream
still writes to memory that the allocator has back: the results are those of a call alone."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8, routing
from int4_weight_only_moe_gb300.layer import MoELayer
from tests.gpu_helpers import Problem, dev
from tests.test_gpu_fp8 import _built, expert, operands, rand  # noqa: F401 (_built: a fixture)

pytestmark = pytest.mark.gpu


def flat(x):
    return [x] if isinstance(x, torch.Tensor) else list(x)


def check(call, same=torch.equal):
    want = [t.clone() for t in flat(call(None))]
    s = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        torch.cuda._sleep(10_000_000)  # some ms, after which the current stream fills what it had
        for t in want:
            for _ in range(2):
                torch.empty_like(t).fill_(3)
        got = flat(call(s))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_router_quantisers_and_product():
    logits = rand((200, 384), 1, dtype=torch.float32)
    check(lambda s: routing.route_scored(logits, 8, stream=s))
    x, w = rand((300, 2048), 2), rand((512, 1024), 3, 0.05)
    views = lambda q, s: (q.view(torch.uint8), s)
    check(lambda s: views(*fp8.quantize(x, stream=s)))
    check(lambda s: views(*fp8.swiglu_quantize(x, stream=s)))
    check(lambda s: views(*fp8.quantize_weight(w, stream=s)))
    ops = operands(40, 1000, 2048, 4)
    check(lambda s: fp8.matmul(*ops, out_dtype=torch.float32, stream=s))


def test_shared_expert_and_its_workspace():
    w = expert(2048, 256, 5)
    for M in (64, 9000):  # workspace from the library's pool, and from torch
        x = rand((M, 2048), M)
        check(lambda s: fp8.shared_expert(x, *w, stream=s))


def test_layer():
    p = Problem(16, 256, 128, 4)
    try:
        layer = MoELayer(p.moe, expert(256, 128, 6), bias=dev(np.linspace(-0.1, 0.1, 16).astype(np.float32)))
        x, logits = rand((300, 256), 7), rand((300, 16), 8, dtype=torch.float32)
        # (the routed experts' fp32 sums are taken in no fixed order: half an ulp of bf16 either way)
        near = lambda a, b: bool(((a - b).abs().float() <= 2.0 ** -7 * b.abs().max().float()).all())

        def call(s):
            p.moe.workspace = None  # a new workspace as well
            return layer.forward(x, logits, stream=s)

        check(call, near)
    finally:
        p.close()
