"""Tensors of torch's function transforms, which have no storage, raise an error in the Python
calls of the order, gather, combine, gradients and adapters, and the calls go on working."""
import pytest
import torch

from tests.test_gpu_calls import CALLS, _built, tensors  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", CALLS)
def test_tensors_without_storage_raise(name):
    call, used = CALLS[name]
    t = tensors()
    want = call(t)
    want = [w.clone() for w in (want if isinstance(want, tuple) else (want,))]
    tried = 0
    for which in used.split():
        def one(v):
            with pytest.raises((RuntimeError, ValueError)):
                call({**t, which: v})
            return v.sum()
        torch.vmap(one)(torch.stack([t[which], t[which]]))
        if t[which].is_floating_point():
            torch.func.grad(one)(t[which])
            torch.func.vjp(one, t[which])
            tried += 1
    assert tried >= 2
    got = call(t)
    for g, w in zip(got if isinstance(got, tuple) else (got,), want):
        assert torch.equal(g, w)
