"""The Python calls of the operators launch on the current device: a tensor that is
somewhere else is refused before anything is launched. Without a GPU: tensors that only
say where they are, and a library that only counts its calls."""
import pytest
import torch

from int4_weight_only_moe_gb300 import fp8, routing

F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


class Tensor:
    def __init__(self, dtype, *shape):
        self.dtype, self.shape, self.dev = dtype, torch.Size(shape), 0

    @property
    def is_cuda(self):
        return self.dev >= 0

    @property
    def device(self):
        return f"cuda:{self.dev}" if self.dev >= 0 else "cpu"

    def get_device(self):
        return self.dev

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[1], 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 256

    @property
    def nbytes(self):
        return 1 << 20


CALLS = {
    "route": (lambda t: routing.route_scored(t["logits"], 2, bias=t["bias"], ids=t["ids"], weights=t["w"]),
              dict(logits=(F32, 4, 64), bias=(F32, 64), ids=(I32, 4, 2), w=(F32, 4, 2))),
    "quantize": (lambda t: fp8.quantize(t["x"], q=t["q"], s=t["s"]),
                 dict(x=(BF16, 4, 256), q=(U8, 4, 256), s=(F32, 4, 2))),
    "swiglu": (lambda t: fp8.swiglu_quantize(t["x"], q=t["q"], s=t["s"]),
               dict(x=(BF16, 4, 512), q=(U8, 4, 256), s=(F32, 4, 2))),
    "weight": (lambda t: fp8.quantize_weight(t["x"], q=t["q"], s=t["s"]),
               dict(x=(BF16, 256, 256), q=(U8, 256, 256), s=(F32, 2, 2))),
    "matmul": (lambda t: fp8.matmul(t["a"], t["a_s"], t["b"], t["b_s"], add=t["add"], out=t["out"]),
               dict(a=(U8, 4, 256), a_s=(F32, 4, 2), b=(U8, 128, 256), b_s=(F32, 1, 2), add=(BF16, 4, 128),
                    out=(BF16, 4, 128))),
    "shared": (lambda t: fp8.shared_expert(t["x"], t["w1"], t["w1_s"], t["w2"], t["w2_s"], add=t["add"], out=t["out"],
                                           workspace=t["ws"]),
               dict(x=(BF16, 4, 256), w1=(U8, 256, 256), w1_s=(F32, 2, 2), w2=(U8, 256, 128), w2_s=(F32, 2, 1),
                    add=(BF16, 4, 256), out=(BF16, 4, 256), ws=(U8, 1 << 20))),
}


@pytest.fixture
def launches(monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    for module in (fp8, routing):
        monkeypatch.setattr(module, "lib", Lib)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    return seen


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_has_to_be_on_the_current_device(launches, name):
    call, shapes = CALLS[name]
    new = lambda: {k: Tensor(*v) for k, v in shapes.items()}
    call(new())
    assert len(launches) == 1
    for which in shapes:
        for dev in (1, -1):
            t = new()
            t[which].dev = dev
            with pytest.raises(ValueError):
                call(t)
    t = new()
    for x in t.values():
        x.dev = 1  # all together on a device that is not the current one
    with pytest.raises(ValueError, match="current device"):
        call(t)
    assert len(launches) == 1


def test_plain_binding_without_a_workspace(launches, monkeypatch):
    import int4_weight_only_moe_gb300 as pkg
    seen = {}

    class Lib:
        def moe_w4a16_shared_expert(self, *args):
            seen["args"] = args
            return 0

    monkeypatch.setattr(pkg, "lib", Lib)
    t = {k: Tensor(*v) for k, v in CALLS["shared"][1].items()}
    pkg.moe_w4a16_shared_expert(t["x"], t["w1"], t["w1_s"], t["w2"], t["w2_s"], None, t["out"], 4, 256, 128, None, stream=0)
    assert seen["args"][5] == 0 and seen["args"][7:12] == (4, 256, 128, 0, 0)
