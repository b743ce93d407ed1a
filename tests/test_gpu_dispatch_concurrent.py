"""Order, gather, combine, gradients and adapters at once on several streams, behind and beside
the 8-bit products whose waits and tensor memory they share, and at sizes whose offsets pass 32
bits. Results are the same bits as one after another."""
import numpy as np
import pytest
import torch

from int4_weight_only_moe_gb300 import dispatch, fp8, lora, routing

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def adapters(M, K, N, r, L, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    return (rand(M, K), rand(L, r, K), rand(L, N, r), torch.randint(-1, L, (M,), generator=g, device="cuda", dtype=torch.int32),
            rand(M, N))


def test_at_once_on_several_streams():
    jobs = []
    for i, (M, K, N, r, L) in enumerate([(3, 2048, 1024, 16, 4), (1000, 1024, 640, 64, 5), (3000, 512, 1024, 32, 9), (600, 2048, 512, 8, 64),
                                         (2000, 768, 384, 128, 2)]):
        x, a, b, index, add = adapters(M, K, N, r, L, i)
        jobs.append(lambda x=x, a=a, b=b, index=index, add=add: (lora.apply(x, a, b, index, add=add),))
    for i, (M, N, K) in enumerate([(40, 1024, 2048), (2048, 1024, 1024)]):
        x, w = torch.randn(M, K, device="cuda", dtype=BF16), torch.randn(N, K, device="cuda", dtype=BF16)
        q, s = fp8.quantize(x)
        b, b_s = fp8.quantize_weight(w)
        jobs.append(lambda q=q, s=s, b=b, b_s=b_s: (fp8.matmul(q, s, b, b_s),))
    for M, E, topk in ((50, 64, 8), (2000, 96, 4)):
        x, l = torch.randn(M, 512, device="cuda", dtype=BF16), torch.randn(M, E, device="cuda")

        def chain(x=x, l=l, E=E, topk=topk):
            ids, w = routing.route_scored(l, topk)
            rows, order = dispatch.sort_gather(x, ids, E, 16)
            out = dispatch.combine(rows, w, order)
            dy, dw = dispatch.combine_backward(x, rows, w, order)
            return out, dw, dispatch.gather_backward(dy, order), routing.route_scored_backward(dw, l, ids)
        jobs.append(chain)
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = []
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(j())
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            for a, b in zip(w, g):
                assert torch.equal(a, b)
    assert fp8.status() == 0


def test_one_behind_the_other():
    """Each call's inputs are the outputs of the one in front of it, written in place again and
    again: a kernel that starts early must wait for them."""
    M, K, E, topk = 700, 512, 32, 4
    x0, l = torch.randn(M, K, device="cuda", dtype=BF16), torch.randn(M, E, device="cuda")
    ids, w = routing.route_scored(l, topk)
    _, a, b, index, _ = adapters(M, K, K, 16, 3, 1)
    a, b = a * K ** -0.5 * 0.1, b * 0.1
    rows, order = dispatch.sort_gather(x0, ids, E, 8)

    def run(sync):
        x, r, o = x0.clone(), torch.zeros_like(rows), dispatch.Order(*(torch.empty_like(t) for t in order))
        for _ in range(20):
            dispatch.sort_gather(x, ids, E, 8, out=r, order=o)
            sync()
            dispatch.combine(r, w, o, add=x, out=x)
            sync()
            lora.apply(x.clone(), a, b, index, add=x, out=x)
            sync()
            dispatch.sort(ids, E, 8, order=o)
            sync()
            dispatch.gather(x, o, out=r)
            sync()
            dispatch.gather_backward(r, o, out=x)
            sync()
            x.mul_(0.2)
        return x

    assert torch.equal(run(lambda: None), run(torch.cuda.synchronize))


@pytest.mark.parametrize("M", [33, 200])
def test_more_adapters_than_rows(M):
    x, a, b, _, add = adapters(M, 264, 72, 12, 1023, 3)
    index = torch.arange(1023 - M, 1023, device="cuda", dtype=torch.int32)
    got = lora.apply(x, a, b, index, add=add, out_dtype=torch.float32).double()
    v = torch.einsum("mk,mrk->mr", x.double(), a[index.long()].double())
    want = add.double() + torch.einsum("mr,mnr->mn", v, b[index.long()].double())
    size = add.double().abs() + torch.einsum("mr,mnr->mn", torch.einsum("mk,mrk->mr", x.double().abs(), a[index.long()].double().abs()),
                                             b[index.long()].double().abs())
    # (K / 16 + 24 and 3 r / 8 + 8 steps of 2^-23, and the output's rounding: see test_gpu_lora.py)
    assert ((got - want).abs() <= (264 / 16 + 24 + 12.5 + 2) * 2.0 ** -23 * size).all()


def test_adapters_beyond_32_bit_offsets():
    M, K, N, r, L = 270_000, 64, 8192, 8, 3   # 2.2e9 outputs
    x, a, b, index, _ = adapters(M, K, N, r, L, 5)
    out = lora.apply(x, a, b, index)
    at = torch.cat([torch.arange(0, 40, device="cuda"), torch.arange(M - 40, M, device="cuda")])
    want = lora.apply(x[at].contiguous(), a, b, index[at].contiguous())
    # (another kernel, whose sums have another order; both round to bf16)
    size = torch.einsum("mk,mrk->mr", x[at].float().abs(), a[index[at].clamp_min(0).long()].float().abs())
    size = torch.einsum("mr,mnr->mn", size, b[index[at].clamp_min(0).long()].float().abs())
    assert ((out[at].float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2 * 40 * 2.0 ** -23 * size).all()
    none = index < 0
    assert not out[none][:100].any()


def test_router_gradient_beyond_32_bit_offsets():
    M, E, topk = 2_200_000, 1000, 4
    l = torch.zeros(M, E, dtype=BF16, device="cuda")
    tail = torch.randn(5, E, device="cuda").to(BF16)
    l[-5:] = tail
    ids = torch.arange(topk, device="cuda", dtype=torch.int32).repeat(M, 1)
    g = torch.ones(M, topk, device="cuda")
    g[-5:] = torch.randn(5, topk, device="cuda")
    for scoring, renorm in (("sigmoid", True), ("softmax", False)):
        got = routing.route_scored_backward(g, l, ids, scoring=scoring, renormalize=renorm)
        want = routing.route_scored_backward(g[-5:].contiguous(), tail, ids[-5:].contiguous(), scoring=scoring, renormalize=renorm)
        assert torch.equal(got[-5:], want) and (got[0] == got[1]).all()
        del got


def test_a_padded_batch():
    """Tokens behind the last real one are marked by ids and adapters of -1, as a batch of a fixed
    size captured into a graph has them."""
    M, real, K, E, topk = 64, 37, 256, 16, 4
    x, l = torch.randn(M, K, device="cuda", dtype=BF16), torch.randn(M, E, device="cuda")
    ids, w = routing.route_scored(l, topk)
    ids[real:] = -1
    x[real:], w[real:] = float("nan"), float("nan")
    rows, order = dispatch.sort_gather(x, ids, E, 8)
    n = int(order.offsets[-1])
    assert rows[:n].isfinite().all() and (order.position[real:] == -1).all()
    out = dispatch.combine(rows, w, order)
    assert out[:real].isfinite().all() and not out[real:].any()
    few, few_order = dispatch.sort_gather(x[:real], ids[:real].contiguous(), E, 8)
    assert torch.equal(out[:real], dispatch.combine(few, w[:real].contiguous(), few_order))
    _, a, b, index, _ = adapters(M, K, 128, 16, 3, 7)
    index[real:] = -1
    add = torch.randn(M, 128, device="cuda", dtype=BF16)
    got = lora.apply(x, a, b, index, add=add)
    assert torch.equal(got[real:], add[real:])
    assert got[:real].isfinite().all()


def test_gradients_of_a_token_with_one_expert_twice():
    x = torch.randn(3, 64, device="cuda")
    ids = torch.tensor([[2, 2], [0, 2], [1, 1]], device="cuda", dtype=torch.int32)
    w = torch.rand(3, 2, device="cuda")
    rows, order = dispatch.sort_gather(x, ids, 3)
    assert order.position.flatten().sort().values.tolist() == list(range(6))
    out = dispatch.combine(rows, w, order)
    np.testing.assert_allclose(out.cpu(), (x * w.sum(1, keepdim=True)).cpu(), rtol=4 * 2.0 ** -24, atol=0)
    dy, dw = dispatch.combine_backward(x, rows, w, order)
    np.testing.assert_allclose(dw.cpu(), (x * x).sum(1, keepdim=True).expand(3, 2).cpu(), rtol=64 * 2.0 ** -24)
