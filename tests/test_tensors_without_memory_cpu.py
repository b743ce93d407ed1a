"""A tensor without memory (one that a function transform made, whose address is 0) is refused
where a tensor may be left out: a 0 there stands for a tensor that is not given, and the call
would go on without its values. Without a GPU: tensors that only say where they are."""
import pytest
import torch

from int4_weight_only_moe_gb300 import dispatch, fp8, lora, routing
from tests.test_dispatch_devices_cpu import CALLS as NEW
from tests.test_dispatch_devices_cpu import calls, launches, new  # noqa: F401 (fixtures)
from tests.test_ops_devices_cpu import CALLS as OLD
from tests.test_ops_devices_cpu import Tensor


class Nowhere(Tensor):
    def data_ptr(self):
        return 0

    def numel(self):
        return self.shape.numel()

    def __len__(self):
        return self.shape[0]


@pytest.mark.parametrize("name,which", [("combine", "w"), ("combine", "add"), ("lora", "add"), ("lora", "scale")])
def test_optional_tensors(calls, name, which):  # noqa: F811
    t = new(name)
    call, shapes, _ = NEW[name]
    call(t)
    assert len(calls) == 1
    t[which] = Nowhere(*shapes[which])
    with pytest.raises(ValueError, match="without memory"):
        call(t)
    assert len(calls) == 1
    t[which] = Nowhere(torch.float32, 0)  # (empty ones have no memory either: their shape is wrong here)
    with pytest.raises(ValueError, match="shape"):
        call(t)


@pytest.mark.parametrize("name,which", [("route", "bias"), ("matmul", "add"), ("shared", "add")])
def test_optional_tensors_of_the_other_operators(launches, monkeypatch, name, which):  # noqa: F811
    call, shapes = OLD[name][:2]
    t = {k: Tensor(*v) for k, v in shapes.items()}
    call(t)
    before = len(launches)
    t[which] = Nowhere(*shapes[which])
    with pytest.raises(ValueError, match="without memory"):
        call(t)
    assert len(launches) == before


def test_empty_tensors_are_not_refused():
    assert routing._dense(torch.zeros(0, 4), torch.float32, (0, 4), "x", -1) == 0
    assert {dispatch._dense, lora._dense, fp8._dense} == {routing._dense}
