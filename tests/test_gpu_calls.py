"""The compiled Python calls give what the Python code's steps give, and refuse what those
refuse: every tensor of a call in turn with another type, shape, layout or device."""
import pytest
import torch

from int4_weight_only_moe_gb300 import MoeW4A16Error, _calls, dispatch, lora, routing

pytestmark = pytest.mark.gpu

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
M, K, E, TOPK = 12, 64, 6, 2


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()
    assert _calls.load() is not None


def tensors():
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s, dtype=F32: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    ids = torch.randint(0, E, (M, TOPK), generator=g, device="cuda", dtype=I32)
    order = dispatch.sort(ids, E, 4)
    R = order.slots.numel()
    return dict(x=rand(M, K, dtype=BF16), ids=ids, offsets=order.offsets, slots=order.slots, position=order.position,
                rows=torch.zeros(R, K, device="cuda", dtype=BF16), y=rand(R, K, dtype=BF16), w=rand(M, TOPK), add=rand(M, K, dtype=BF16),
                out=torch.zeros(M, K, device="cuda", dtype=BF16), g=rand(M, K), dy=torch.zeros(R, K, device="cuda", dtype=BF16),
                dw=torch.zeros(M, TOPK, device="cuda"), l=rand(M, E), dl=torch.zeros(M, E, device="cuda"),
                a=rand(3, 8, K, dtype=BF16), b=rand(3, 40, 8, dtype=BF16), index=torch.randint(-1, 3, (M,), generator=g, device="cuda", dtype=I32),
                scale=rand(3), lo=torch.zeros(M, 40, device="cuda", dtype=BF16), la=rand(M, 40))


def order(t):
    return dispatch.Order(t["offsets"], t["slots"], t["position"])


CALLS = {
    "gather": (lambda t, **k: dispatch.gather(t["x"], order(t), out=t["rows"], **k), "x offsets slots position rows"),
    "sort_gather": (lambda t, **k: dispatch.sort_gather(t["x"], t["ids"], E, 4, out=t["rows"], order=order(t), **k)[0],
                    "x ids offsets slots position rows"),
    "combine": (lambda t, **k: dispatch.combine(t["y"], t["w"], order(t), add=t["add"], out=t["out"], **k), "y w position add out"),  # (slots: their number only)
    "gather_backward": (lambda t, **k: dispatch.gather_backward(t["y"], order(t), out=t["out"], **k), "y position out"),
    "combine_backward": (lambda t, **k: dispatch.combine_backward(t["g"], t["y"], t["w"], order(t), dy=t["dy"], dweights=t["dw"], **k),
                         "g y w offsets slots position dy dw"),
    "route_backward": (lambda t, **k: routing.route_scored_backward(t["w"], t["l"], t["ids"], out=t["dl"], **k), "w l ids dl"),
    "lora": (lambda t, **k: lora.apply(t["x"], t["a"], t["b"], t["index"], add=t["la"], scale=t["scale"], out=t["lo"], **k),
             "x a b index la scale lo"),
}


@pytest.mark.parametrize("name", CALLS)
def test_same_as_the_python_steps(name):
    call, _ = CALLS[name]
    first, second = tensors(), tensors()
    a = call(first)
    b = call(second, stream=torch.cuda.current_stream())  # (a given stream takes the steps)
    for p, q in zip(a if isinstance(a, tuple) else (a,), b if isinstance(b, tuple) else (b,)):
        assert torch.equal(p, q) and p.any()


@pytest.mark.parametrize("name", CALLS)
def test_every_tensor_is_checked(name):
    call, used = CALLS[name]
    for which in used.split():
        t = tensors()
        v = t[which]
        wrong = [v.cpu(), v.double(), v.unsqueeze(0)]
        if (name, which) != ("gather_backward", "position"):  # (there any number of choices is right)
            wrong.append(torch.cat([v, v], -1))
        if v.dim() > 1:
            wrong.append(torch.cat([v, v], -1)[..., ::2])
        for bad in wrong:
            t[which] = bad
            with pytest.raises((ValueError, MoeW4A16Error)):
                call(t)
    torch.cuda.synchronize()


def test_strided_rows_and_optional_tensors():
    t = tensors()
    wide = torch.randn(2 * M, K + 8, device="cuda").to(BF16)
    x = wide[::2, 8:]
    assert torch.equal(dispatch.gather(x, order(t), out=t["rows"].clone()), dispatch.gather(x.contiguous(), order(t), out=t["rows"].clone()))
    lo = lora.apply(x, t["a"], t["b"], t["index"], out=t["lo"])
    assert torch.equal(lo, lora.apply(x.contiguous(), t["a"], t["b"], t["index"]))
    out = dispatch.combine(t["y"], t["w"], order(t), out=t["out"])
    assert torch.equal(out, dispatch.combine(t["y"], t["w"], order(t)))
    l = torch.randn(M, 2 * E, device="cuda")
    assert torch.equal(routing.route_scored_backward(t["w"], l[:, :E], t["ids"], out=t["dl"]),
                       routing.route_scored_backward(t["w"], l[:, :E].contiguous(), t["ids"]))


def test_errors_of_the_library_are_raised():
    t = tensors()
    with pytest.raises(MoeW4A16Error):
        routing.route_scored_backward(t["w"], t["l"], t["ids"], out=t["l"])
    with pytest.raises(MoeW4A16Error):
        dispatch.combine_backward(t["g"], t["y"], t["w"], order(t), dy=t["y"], dweights=t["dw"])
