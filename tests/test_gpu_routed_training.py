"""The operators around expert products of the caller's own, as a training step uses them:
route, sort and gather, a bf16 SwiGLU expert on each expert's rows (torch), combine; then the
way back to the experts' weights, the hidden states and the router's logits. Against the same
step in 64 bits by autograd, with the same choices.

Tolerance: rows, products and gradients of products are rounded to bf16 on the way (each
half a step, 2^-8 of it), a handful one after another: relative L2 2e-2 = 5 * 2^-8. The
forward rounds the experts' rows and the output: below 3 * 2^-8."""
import pytest
import torch

from int4_weight_only_moe_gb300 import dispatch, routing

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import __graft_entry__
    __graft_entry__.build()


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def expert(x, w1, w2):
    g, u = (x @ w1.t()).chunk(2, 1)
    return torch.nn.functional.silu(g) * u @ w2.t()


@pytest.mark.parametrize("M,E,topk,block", [(64, 8, 2, 1), (257, 16, 4, 16), (1500, 12, 3, 128)])
@pytest.mark.parametrize("scoring,renormalize", [("sigmoid", True), ("softmax", False)])
def test_step(M, E, topk, block, scoring, renormalize):
    K, N = 128, 64
    gen = torch.Generator(device="cuda").manual_seed(M)
    rand = lambda *s, by=1.0: torch.randn(*s, generator=gen, device="cuda") * by  # noqa: E731
    x, l = rand(M, K).bfloat16(), rand(M, E)
    w1, w2 = rand(E, 2 * N, K, by=K ** -0.5).bfloat16(), rand(E, K, N, by=N ** -0.5).bfloat16()
    add, dout = rand(M, K).bfloat16(), rand(M, K).bfloat16()

    # ours
    ids, w = routing.route_scored(l, topk, scoring=scoring, renormalize=renormalize, scale=2.5)
    rows, order = dispatch.sort_gather(x, ids, E, block)
    off = order.offsets.tolist()
    y = torch.zeros_like(rows)
    parts = []
    for e in range(E):
        r = rows[off[e]:off[e + 1]].detach().requires_grad_()
        a, b = w1[e].detach().requires_grad_(), w2[e].detach().requires_grad_()
        out_e = expert(r, a, b)
        y[off[e]:off[e + 1]] = out_e.detach()
        parts.append((r, a, b, out_e))
    out = dispatch.combine(y, w, order, add=add)
    dy, dw = dispatch.combine_backward(dout, y, w, order)
    drows = torch.zeros_like(rows)
    for e, (r, a, b, out_e) in enumerate(parts):
        if len(r):
            out_e.backward(dy[off[e]:off[e + 1]])
            drows[off[e]:off[e + 1]] = r.grad
    dx = dispatch.gather_backward(drows, order)
    dl = routing.route_scored_backward(dw, l, ids, scoring=scoring, renormalize=renormalize, scale=2.5)

    # 64 bits, by autograd
    X, Lg = x.double().requires_grad_(), l.double().requires_grad_()
    W1, W2 = w1.double().requires_grad_(), w2.double().requires_grad_()
    s = torch.sigmoid(Lg) if scoring == "sigmoid" else torch.softmax(Lg, 1)
    p = s.gather(1, ids.long())
    W = (p / p.sum(1, keepdim=True) if renormalize else p) * 2.5
    O = add.double()
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        O = O.index_add(0, t, expert(X[t], W1[e], W2[e]) * W[t, j].unsqueeze(1))
    O.backward(dout.double())

    assert rel(out, O.detach()) < 3 * 2.0 ** -8
    assert rel(dx, X.grad) < 2e-2 and rel(dl, Lg.grad) < 2e-2
    for e, (r, a, b, _) in enumerate(parts):
        if (ids == e).any():
            assert rel(a.grad, W1.grad[e]) < 2e-2 and rel(b.grad, W2.grad[e]) < 2e-2


def test_two_halves_of_the_experts_add_up():
    """Expert parallelism: each part sorts, gathers and combines its own experts' rows; the
    parts' fp32 sums add up to the whole, the gradients of their rows and weights are the
    whole's."""
    M, E, topk, K = 300, 24, 4, 64
    x = torch.randn(M, K, device="cuda")
    ids, w = routing.route_scored(torch.randn(M, E, device="cuda"), topk)
    whole, order = dispatch.sort_gather(x, ids, E)
    want = dispatch.combine(whole, w, order)
    dy, dw = dispatch.combine_backward(want, whole, w, order)
    total, dw_total, rows_seen = torch.zeros_like(want), torch.zeros_like(dw), 0
    for part in ((0, 10), (10, 24)):
        rows, mine = dispatch.sort_gather(x, ids, E, expert_range=part)
        n = int(mine.offsets[-1])
        assert torch.equal(rows[:n], whole[rows_seen:rows_seen + n])
        total += dispatch.combine(rows, w, mine)
        d, g = dispatch.combine_backward(want, rows, w, mine)
        assert torch.equal(d[:n], dy[rows_seen:rows_seen + n])
        dw_total += g
        rows_seen += n
    assert rows_seen == M * topk
    assert torch.equal(dw_total, dw)  # (each weight has its gradient from one part, 0 from the other)
    # (two sums of at most four products in place of one: five roundings of 2^-24)
    size = (w.abs() * 1.0).sum(1, keepdim=True) * x.abs()
    assert ((total - want).abs() <= 5 * 2.0 ** -24 * size).all()
