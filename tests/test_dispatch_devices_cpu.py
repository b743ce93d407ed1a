"""The Python calls of the order, gather, combine, gradients and adapters: a tensor that is
not on the current device is refused before anything is launched, and what a call makes for
kernels on a given stream is taken in that stream's order. Without a GPU, as for the other
operators (test_ops_devices_cpu.py, test_new_tensors_cpu.py)."""
import pytest
import torch

import int4_weight_only_moe_gb300 as pkg
from int4_weight_only_moe_gb300 import dispatch, lora, routing
from tests.test_new_tensors_cpu import Stream, made  # noqa: F401 (a fixture)
from tests.test_ops_devices_cpu import Tensor, launches  # noqa: F401 (a fixture)

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
M, K, E, TOPK = 4, 256, 16, 2
ROWS = M * TOPK + min(E, M * TOPK) * 3  # block 4


class T(Tensor):
    def __len__(self):
        return self.shape[0]


def order(t):
    return dispatch.Order(t["offsets"], t["slots"], t["position"])


ORDER = dict(offsets=(I32, E + 1), slots=(I32, ROWS), position=(I32, M, TOPK))
CALLS = {
    "sort": (lambda t, **kw: dispatch.sort(t["ids"], E, 4, order=order(t), **kw), dict(ids=(I32, M, TOPK), **ORDER), 0),
    "gather": (lambda t, **kw: dispatch.gather(t["x"], order(t), out=t["out"], **kw),
               dict(x=(BF16, M, K), out=(BF16, ROWS, K), **ORDER), 0),
    "sort_gather": (lambda t, **kw: dispatch.sort_gather(t["x"], t["ids"], E, 4, out=t["out"], order=order(t), **kw),
                    dict(x=(BF16, M, K), ids=(I32, M, TOPK), out=(BF16, ROWS, K), **ORDER), 0),
    "combine": (lambda t, **kw: dispatch.combine(t["y"], t["w"], order(t), add=t["add"], out=t["out"], **kw),
                dict(y=(BF16, ROWS, K), w=(F32, M, TOPK), add=(BF16, M, K), out=(BF16, M, K), position=(I32, M, TOPK)), 0),
    "combine_backward": (lambda t, **kw: dispatch.combine_backward(t["g"], t["y"], t["w"], order(t), dy=t["dy"], dweights=t["dw"], **kw),
                         dict(g=(BF16, M, K), y=(BF16, ROWS, K), w=(F32, M, TOPK), dy=(BF16, ROWS, K), dw=(F32, M, TOPK), **ORDER), 0),
    "route_backward": (lambda t, **kw: routing.route_scored_backward(t["dw"], t["l"], t["ids"], out=t["out"], **kw),
                       dict(dw=(F32, M, TOPK), l=(F32, M, E), ids=(I32, M, TOPK), out=(F32, M, E)), 0),
    "lora": (lambda t, **kw: lora.apply(t["x"], t["a"], t["b"], t["index"], add=t["add"], scale=t["scale"], out=t["out"],
                                        workspace=t["ws"], **kw),
             dict(x=(BF16, M, K), a=(BF16, 3, 8, K), b=(BF16, 3, 64, 8), index=(I32, M), add=(F32, M, 64), scale=(F32, 3),
                  out=(BF16, M, 64), ws=(U8, 1 << 20)), 0),
}


@pytest.fixture
def calls(monkeypatch, launches):  # noqa: F811
    class Lib:
        def __getattr__(self, name):
            return lambda *a: launches.append(name) or 0

    for module in (dispatch, lora, routing):
        monkeypatch.setattr(module, "lib", Lib)
    monkeypatch.setattr(dispatch, "_order_rows", lambda m, k, e, b: m * k + min(e, m * k) * (b - 1))
    monkeypatch.setattr(lora, "_workspace_size", lambda *a: 0)
    return launches


def new(name):
    t = {k: T(*v) for k, v in CALLS[name][1].items()}
    for k, v in dict(ORDER).items():
        t.setdefault(k, T(*v))
    return t


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_has_to_be_on_the_current_device(calls, name):
    call, shapes, _ = CALLS[name]
    call(new(name))
    assert len(calls) == 1
    for which in shapes:
        for dev in (1, -1):
            t = new(name)
            t[which].dev = dev
            with pytest.raises(ValueError):
                call(t)
    t = new(name)
    for x in t.values():
        x.dev = 1
    with pytest.raises(ValueError, match="current device"):
        call(t)
    assert len(calls) == 1


MADE = {"sort": 3, "gather": 1, "sort_gather": 4, "combine": 1, "combine_backward": 2, "route_backward": 1, "lora": 1}
PLAIN = {
    "sort": lambda t, s: dispatch.sort(t["ids"], E, 4, stream=s),
    "gather": lambda t, s: dispatch.gather(t["x"], order(t), stream=s),
    "sort_gather": lambda t, s: dispatch.sort_gather(t["x"], t["ids"], E, 4, stream=s),
    "combine": lambda t, s: dispatch.combine(t["y"], t["w"], order(t), stream=s),
    "combine_backward": lambda t, s: dispatch.combine_backward(t["g"], t["y"], t["w"], order(t), stream=s),
    "route_backward": lambda t, s: routing.route_scored_backward(t["dw"], t["l"], t["ids"], stream=s),
    "lora": lambda t, s: lora.apply(t["x"], t["a"], t["b"], t["index"], stream=s),
}


@pytest.mark.parametrize("stream,other", [(Stream(9), True), (9, True), (None, False), (7, False)],
                         ids=["stream", "handle", "none", "current"])
@pytest.mark.parametrize("name", PLAIN)
def test_made_on_the_stream_that_writes_them(made, calls, monkeypatch, name, stream, other):  # noqa: F811
    count = MADE[name]
    if name == "lora":  # with a workspace of torch's as well
        monkeypatch.setattr(lora, "_workspace_size", lambda *a: lora._POOL_BYTES + 1)
        count += 1
    PLAIN[name](new(name), stream)
    assert len(made) == count
    for t in made:
        assert t.made_on == (9 if other else 7) and t.recorded == ([7] if other else [])


def test_plain_bindings_pass_what_they_are_given(monkeypatch):
    seen = {}

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.update({name: a}) or 0

    monkeypatch.setattr(pkg, "lib", Lib)
    t = new("lora")
    pkg.moe_w4a16_lora(t["x"], K, t["a"], t["b"], None, t["index"], None, 0, t["out"], 1, M, K, 64, 8, 3, None, stream=0)
    assert seen["moe_w4a16_lora"] == (256, K, 256, 256, 0, 256, 0, 0, 256, 1, M, K, 64, 8, 3, 0, 0, 0)
    t = new("combine_backward")
    pkg.moe_w4a16_combine_backward(t["g"], 1, t["y"], 1, t["w"], *order(t), t["dy"], t["dw"], M, K, TOPK, E, 4, stream=0)
    args, types = seen["moe_w4a16_combine_backward"], pkg._SIGNATURES["moe_w4a16_combine_backward"][1]
    assert len(args) == len(types)
    for name, call in (("sort", lambda t: pkg.moe_w4a16_dispatch_sort(t["ids"], M, TOPK, 0, E, 4, *order(t), stream=0)),
                       ("gather", lambda t: pkg.moe_w4a16_dispatch_gather(t["x"], 1, K, *order(t), t["out"], M, K, TOPK, E, 4, stream=0)),
                       ("sort_gather", lambda t: pkg.moe_w4a16_dispatch_sort_gather(t["x"], 1, K, t["ids"], M, K, TOPK, 0, E, 4,
                                                                                    *order(t), t["out"], stream=0)),
                       ("combine", lambda t: pkg.moe_w4a16_combine(t["y"], 1, t["w"], t["position"], t["add"], t["out"], 1, M, K,
                                                                   TOPK, ROWS, stream=0)),
                       ("route_backward", lambda t: pkg.moe_w4a16_route_scored_backward(t["dw"], t["l"], 0, E, t["ids"], M, E, TOPK,
                                                                                        1, True, 1.0, t["out"], stream=0))):
        seen.clear()
        call(new(name))
        (fn, args), = seen.items()
        assert len(args) == len(pkg._SIGNATURES[fn][1]), fn
