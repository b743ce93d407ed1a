"""The compiled Python calls without a GPU: they take no tensor that is not on the device, nor
anything else that is not plainly a tensor, and leave those to the Python code."""
import pytest
import torch

NAMES = {"gather": 7, "sort_gather": 11, "combine": 8, "combine_backward": 10, "route_backward": 9, "lora": 10}


@pytest.fixture(scope="module")
def calls():
    import __graft_entry__
    __graft_entry__.build()
    from int4_weight_only_moe_gb300 import _calls
    m = _calls.load()
    assert m is not None and _calls.load() is m and _calls.module is m
    return m


ARGS = {  # (what stands behind device and stream, in order)
    "gather": "t t t t t", "sort_gather": "t t 4 0 1 t t t t", "combine": "t t t t t t", "combine_backward": "t t t t t t t t",
    "route_backward": "t t t 1 1 1.0 t", "lora": "t t t t t t t 0"}


@pytest.mark.parametrize("name", NAMES)
def test_leaves_what_is_not_its_own(calls, name):
    class Subclass(torch.Tensor):
        pass

    for what in (torch.zeros(4, 4), torch.zeros(4, 4).as_subclass(Subclass), None, 7, "x", torch.nn.Parameter(torch.zeros(4, 4)),
                 torch.zeros(4, 4).to_sparse(), torch.zeros(4, 4, device="meta")):
        args = [what if a == "t" else float(a) if "." in a else int(a) for a in ARGS[name].split()]
        assert len(args) == NAMES[name] - 2
        assert getattr(calls, name)(0, 0, *args) is None


@pytest.mark.parametrize("name", NAMES)
def test_refuses_another_number_of_arguments(calls, name):
    for n in (0, NAMES[name] - 1, NAMES[name] + 1):
        with pytest.raises(TypeError):
            getattr(calls, name)(*[0] * n)


def test_numbers_that_are_none(calls):
    t = torch.zeros(4, 4)
    with pytest.raises(TypeError):
        calls.sort_gather(0, 0, t, t, 4.5, 0, 1, t, t, t, t)
    with pytest.raises((TypeError, OverflowError)):
        calls.sort_gather(0, 0, t, t, 1 << 80, 0, 1, t, t, t, t)
    with pytest.raises(TypeError):
        calls.route_backward(0, 0, t, t, t, 1, True, "x", t)
    with pytest.raises(TypeError):
        calls.lora("device", 0, t, t, t, t, t, t, t, 0)


def test_a_library_that_is_not_built_leaves_everything_to_python(monkeypatch):
    from int4_weight_only_moe_gb300 import _calls, routing
    monkeypatch.setattr(_calls, "module", None)
    monkeypatch.setattr(_calls, "PATH", "/nonexistent/moe_w4a16_calls.so")
    assert _calls.load() is None
    assert routing._fast(torch.zeros(2, 2)) is None
