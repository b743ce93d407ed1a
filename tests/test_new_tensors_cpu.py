"""Outputs and workspaces that a call makes for kernels on a given stream are taken in that
stream's order, and kept until the caller's current stream is done with them. Without a GPU:
the allocator and the streams are recorders."""
import contextlib

import pytest
import torch

import int4_weight_only_moe_gb300 as pkg
from int4_weight_only_moe_gb300 import fp8, routing
from tests.test_ops_devices_cpu import CALLS, Tensor, launches  # noqa: F401 (launches: a fixture)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class Made(Tensor):
    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


@pytest.fixture
def made(monkeypatch, launches):  # noqa: F811
    current, out = [Stream(7)], []

    @contextlib.contextmanager
    def on(s):
        current.append(s)
        yield
        current.pop()

    def empty(shape, dtype, device):
        t = Made(dtype, *shape)
        t.made_on, t.recorded = current[-1].cuda_stream, []
        out.append(t)
        return t

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current[-1])
    monkeypatch.setattr(torch, "empty", empty)
    return out


def call(name, stream):
    t = {k: Tensor(*v) for k, v in CALLS[name][1].items()}
    if name == "route":
        return routing.route_scored(t["logits"], 2, stream=stream)
    if name == "matmul":
        return fp8.matmul(t["a"], t["a_s"], t["b"], t["b_s"], stream=stream)
    if name == "shared":
        return fp8.shared_expert(t["x"], t["w1"], t["w1_s"], t["w2"], t["w2_s"], stream=stream)
    return {"quantize": fp8.quantize, "swiglu": fp8.swiglu_quantize, "weight": fp8.quantize_weight}[name](
        t["x"], stream=stream)


@pytest.mark.parametrize("stream", [Stream(9), 9], ids=["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_made_on_the_stream_that_writes_them(made, monkeypatch, name, stream):
    if name == "shared":  # with a workspace of torch's as well
        monkeypatch.setattr(fp8, "_workspace_size", lambda *a: fp8._POOL_BYTES + 1)
    call(name, stream)
    assert len(made) == (1 if name == "matmul" else 2)
    for t in made:
        assert t.made_on == 9 and t.recorded == [7]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream", [None, 7])
def test_the_current_stream_needs_nothing(made, monkeypatch, name, stream):
    monkeypatch.setattr(fp8, "_workspace_size", lambda *a: 256)
    call(name, stream)
    assert made and all(t.made_on == 7 and not t.recorded for t in made)


def test_a_workspace_that_grows(made, monkeypatch):
    monkeypatch.setattr(pkg, "moe_w4a16_workspace_size", lambda h, M: 1000 * M)
    moe = pkg.MoEW4A16.__new__(pkg.MoEW4A16)
    moe.handle, moe.workspace = None, None
    Made.numel = lambda self: self.shape[0]
    first = moe.ensure_workspace(1, stream=9)
    assert first.made_on == 9 and first.recorded == [7]
    second = moe.ensure_workspace(2, stream=11)  # a call of stream 11 may still use the first
    assert second.made_on == 11 and first.recorded == [7, 11]
    assert moe.ensure_workspace(2) is second
