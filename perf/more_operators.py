"""Measured cases of the operators between the router and the experts, and beside the
projections: tokens sorted by expert and back with their weights, the gradients of both
and of the router, and low-rank adapters of many requests.

``run`` computes each in elementary torch operations (fp32, rounded once at the end) or,
where ``own`` is true, with the library's kernels. Definitions, with slot i = t * topk + j
standing for token t's j-th choice:

* dispatch       rows = the slots by expert, then by slot, an expert's rows filled up to a
                 multiple of ``block``; offsets = where each expert's begin; slots = the slot
                 of a row (-1: none); position = the row of a slot (-1: the id is no expert);
                 out[row] = x[token of the row], 0 in rows that fill up; rows behind the last
                 expert's are left as they were.
* dispatch_grad  dx[t] = sum_j dout[position[t, j]].
* combine        out[t] = sum_j w[t, j] y[position[t, j]] (+ add[t]).
* combine_grad   dy[position[t, j]] = w[t, j] g[t] (0 in rows that fill up),
                 dw[t, j] = <g[t], y[position[t, j]]>.
* route_grad     gradient of the router's weights (scores of the chosen ids, divided by their
                 sum if ``renorm``, times ``scale``) with regard to the logits.
* lora           out[m] = add[m] + scale[l] b[l] (a[l] x[m]) with l = index[m]; out[m] = add[m]
                 where that is -1.
"""
import math

import torch

own = False


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # a decode step of four requests through the layer of this framework's benchmark
        # (384 experts, top-8, 7,168 wide)
        dict(name="dispatch_decode", op="dispatch", M=4, K=7168, E=384, topk=8, block=1, drop=0.0, dtype="bfloat16"),
        # a prompt of 8,192 tokens, each expert's rows filled up to whole tiles of 128
        dict(name="dispatch_prompt", op="dispatch", M=8192, K=7168, E=384, topk=8, block=128, drop=0.0,
             dtype="bfloat16"),
        # a training chunk of odd length, some choices dropped: hidden states' gradient
        dict(name="dispatch_grad_chunk", op="dispatch_grad", M=2047, K=2048, E=160, topk=6, block=16, drop=0.02,
             dtype="bfloat16"),
        # a verify batch: experts' rows back to the tokens, added to the shared expert's output
        dict(name="combine_verify", op="combine", M=90, K=7168, E=384, topk=8, block=1, drop=0.0, add=True,
             dtype="bfloat16"),
        # the prompt's experts' rows back to the tokens
        dict(name="combine_prompt", op="combine", M=8192, K=7168, E=384, topk=8, block=128, drop=0.0, add=False,
             dtype="bfloat16"),
        # gradients of a small training batch, fp32 rows; and of a long one
        dict(name="combine_grad_small", op="combine_grad", M=333, K=2048, E=64, topk=6, block=1, drop=0.0,
             dtype="float32"),
        dict(name="combine_grad_prompt", op="combine_grad", M=4096, K=7168, E=384, topk=8, block=128, drop=0.0,
             dtype="bfloat16"),
        # the router of a long training batch; and one with softmax scores taken as they are
        dict(name="route_grad_prompt", op="route_grad", M=16384, E=384, topk=8, scoring="sigmoid", renorm=True,
             scale=2.5, dtype="float32"),
        dict(name="route_grad_softmax", op="route_grad", M=4097, E=160, topk=6, scoring="softmax", renorm=False,
             scale=16.0, dtype="bfloat16"),
        # one request's token beside the shared expert's gate/up product, whose fp32 sums it joins
        dict(name="lora_decode", op="lora", M=1, K=7168, N=4096, r=16, L=8, none=0.0, mixed=True, add="float32"),
        # a decode batch of many requests, 32 adapters, some requests without one
        dict(name="lora_batch", op="lora", M=64, K=7168, N=4096, r=32, L=32, none=0.1, mixed=True, add="float32"),
        # prompts of several requests one after another beside the product's bf16 output
        dict(name="lora_prompt", op="lora", M=8192, K=7168, N=4096, r=64, L=8, none=0.05, mixed=False,
             add="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine", "combine_grad", "route_grad", "lora", "lora"])
    if op == "route_grad":
        E = _log_int(rng, 8, 384)
        scoring = rng.choice(["sigmoid", "softmax"])
        return dict(op=op, M=_log_int(rng, 1, 16384), E=E, topk=rng.randint(1, min(E, 12)), scoring=scoring,
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, 16.0]),
                    dtype=rng.choice(["float32", "bfloat16"]))
    if op == "lora":
        return dict(op=op, M=_log_int(rng, 1, 8192), K=8 * _log_int(rng, 32, 896), N=8 * _log_int(rng, 32, 512),
                    r=8 * rng.randint(1, 8), L=_log_int(rng, 1, 48), none=rng.choice([0.0, 0.05, 0.3]),
                    mixed=rng.random() < 0.5, add=rng.choice(["float32", "bfloat16", "bfloat16"]))
    E = _log_int(rng, 8, 384)
    dtype = rng.choice(["float32", "bfloat16", "bfloat16"])
    most = {"dispatch": 8192, "dispatch_grad": 8192, "combine": 8192, "combine_grad": 4096}[op]
    case = dict(op=op, M=_log_int(rng, 1, most // (2 if dtype == "float32" else 1)), K=8 * _log_int(rng, 32, 896), E=E,
                topk=rng.randint(1, 8), block=rng.choice([1, 1, 16, 128]), drop=rng.choice([0.0, 0.0, 0.05]), dtype=dtype)
    if op == "combine":
        case["add"] = rng.random() < 0.5
    return case


def _capacity(case):
    slots = case["M"] * case["topk"]
    return slots + min(case["E"], slots) * (case["block"] - 1)


def work(case):
    M, op = case["M"], case["op"]
    if op == "route_grad":
        E, k = case["E"], case["topk"]
        item = 4 if case["dtype"] == "float32" else 2
        read = E * item if case["scoring"] == "softmax" and not case["renorm"] else k * item
        return {"bytes": M * (E * item + read + 8 * k), "flops": 0}
    if op == "lora":
        K, N, r = case["K"], case["N"], case["r"]
        used = min(case["L"], max(1, int(M * (1.0 - case["none"]))))
        return {"bytes": M * K * 2 + M * N * (2 + (4 if case["add"] == "float32" else 2)) + used * r * (K + N) * 2 + 4 * M,
                "flops": 2 * M * r * (K + N)}
    K, slots = case["K"], case["M"] * case["topk"]
    item = 4 if case["dtype"] == "float32" else 2
    rows = slots * (1.0 - case["drop"])
    if op == "dispatch":
        return {"bytes": (M + rows) * K * item + 4 * (2 * slots + _capacity(case) + case["E"]), "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": (M + rows) * K * item + 4 * slots, "flops": rows * K}
    if op == "combine":
        return {"bytes": (M * (2 if case["add"] else 1) + rows) * K * item + 8 * slots, "flops": 2 * rows * K}
    return {"bytes": (M + 2 * rows) * K * item + 12 * slots, "flops": 3 * rows * K}


# ----------------------------------------------------------------------------- inputs


def _choices(gen, M, E, topk, drop):
    """Expert ids [M, topk], different ones for a token (as far as there are), some experts
    several times as busy as others; a share ``drop`` of them -1."""
    busy = torch.randn(E, generator=gen, device="cuda") * 0.7
    l = busy + torch.randn(M, max(E, topk), generator=gen, device="cuda")[:, :E]
    if topk > E:
        l = l.repeat(1, -(-topk // E))
    ids = (torch.topk(l, topk, dim=1).indices % E).to(torch.int32)
    if drop:
        ids = torch.where(torch.rand(M, topk, generator=gen, device="cuda") < drop, -1, ids)
    return ids.contiguous()


def _order(ids, E, block, capacity):
    """(offsets [E + 1], slots [capacity], position [M, topk]) of expert ids."""
    flat = ids.reshape(-1).long()
    n = flat.numel()
    known = (flat >= 0) & (flat < E)
    key = torch.where(known, flat, E)
    sorted_key, by = torch.sort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    first = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + block - 1) // block * block
    offsets = torch.cat([torch.zeros_like(padded[:1]), torch.cumsum(padded, 0)])
    row = offsets[sorted_key] + torch.arange(n, device=ids.device) - first[sorted_key]
    row = torch.where(sorted_key < E, row, capacity)  # (one more place, for what is no expert's)
    slots = torch.full((capacity + 1,), -1, dtype=torch.int32, device=ids.device)
    slots = slots.scatter(0, row, by.to(torch.int32))[:capacity]
    position = torch.empty(n, dtype=torch.int32, device=ids.device)
    position = position.scatter(0, by, torch.where(sorted_key < E, row, -1).to(torch.int32))
    return offsets.to(torch.int32), slots.contiguous(), position.view(ids.shape)


def _hidden(gen, *shape):
    """Hidden states: normal, a few channels several times the rest."""
    x = torch.randn(*shape, generator=gen, device="cuda")
    gain = torch.ones(shape[-1], device="cuda")
    gain[torch.randint(0, shape[-1], (max(1, shape[-1] // 200),), generator=gen, device="cuda")] = 8.0
    return x.mul_(gain)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    M, op = case["M"], case["op"]
    st = dict(case=dict(case))
    new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if op == "route_grad":
        E, k = case["E"], case["topk"]
        dtype = getattr(torch, case["dtype"])
        st["logits"] = (rand(M, E) * 1.5).to(dtype)
        c = st["logits"].float() + (rand(E) * 0.3 if case["scoring"] == "sigmoid" else 0.0)
        st["ids"] = torch.topk(c, k, dim=1).indices.to(torch.int32).contiguous()
        st["g"] = rand(M, k) * 0.1
        st["out"] = new(M, E, dtype=dtype)
        return st
    if op == "lora":
        K, N, r, L = case["K"], case["N"], case["r"], case["L"]
        st["x"] = _hidden(gen, M, K).to(torch.bfloat16)
        st["a"] = (rand(L, r, K) * K ** -0.5).to(torch.bfloat16)
        st["b"] = (rand(L, N, r) * r ** -0.5).to(torch.bfloat16)
        st["scale"] = torch.rand(L, generator=gen, device="cuda") + 0.5
        if case["mixed"]:  # requests of one token each
            index = torch.randint(0, L, (M,), generator=gen, device="cuda")
            index = torch.where(torch.rand(M, generator=gen, device="cuda") < case["none"], -1, index)
        else:  # requests of many tokens, one after another
            n = max(1, min(M, 2 * L))
            ends = torch.sort(torch.rand(n, generator=gen, device="cuda")).values
            which = torch.searchsorted(ends, (torch.arange(M, device="cuda") + 0.5) / M)
            of = torch.randint(0, L, (n + 1,), generator=gen, device="cuda")
            of = torch.where(torch.rand(n + 1, generator=gen, device="cuda") < case["none"], -1, of)
            index = of[which]
        st["index"] = index.to(torch.int32).contiguous()
        st["add"] = (rand(M, N) * 2.0).to(getattr(torch, case["add"]))
        st["out"] = new(M, N, dtype=torch.bfloat16)
        return st
    K, E, k, dtype = case["K"], case["E"], case["topk"], getattr(torch, case["dtype"])
    capacity = _capacity(case)
    st["ids"] = _choices(gen, M, E, k, case["drop"])
    if op == "dispatch":
        st["x"] = _hidden(gen, M, K).to(dtype)
        # (rows behind the last expert's stay what they are: the tests of equality want a value)
        st["out"] = torch.zeros(capacity, K, dtype=dtype, device="cuda")
        st["order"] = (new(E + 1, dtype=torch.int32), new(capacity, dtype=torch.int32), new(M, k, dtype=torch.int32))
        return st
    st["order"] = _order(st["ids"], E, case["block"], capacity)
    st["w"] = torch.softmax(rand(M, k), 1) * 2.5
    if op == "combine":
        st["y"] = _hidden(gen, capacity, K).to(dtype)
        st["add"] = rand(M, K).to(dtype) if case["add"] else None
        st["out"] = new(M, K, dtype=dtype)
    elif op == "dispatch_grad":
        st["dout"] = (rand(capacity, K) * 0.1).to(dtype)
        st["out"] = new(M, K, dtype=dtype)
    else:
        st["y"] = _hidden(gen, capacity, K).to(dtype)
        st["g"] = (rand(M, K) * 0.1).to(dtype)
        st["out"] = (torch.zeros(capacity, K, dtype=dtype, device="cuda"), new(M, k, dtype=torch.float32))
    return st


# ------------------------------------------------------------------------------- runs


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _rows_of(t, position):
    """t[position] in fp32, zeros where that is -1."""
    found = t[position.clamp_min(0).long()].float()
    return torch.where((position >= 0).unsqueeze(-1), found, torch.zeros((), device=t.device))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route_grad":
        l, ids, g = st["logits"].float(), st["ids"].long(), st["g"]
        if case["scoring"] == "sigmoid":
            s = 1.0 / (1.0 + torch.exp(-l))
        else:
            e = torch.exp(l - l.amax(-1, keepdim=True))
            s = e / e.sum(-1, keepdim=True)
        p = s.gather(1, ids)
        if case["renorm"]:
            total = p.sum(-1, keepdim=True)
            u = (g - (g * p).sum(-1, keepdim=True) / total) / total
        else:
            u = g
        ds = torch.zeros_like(s).scatter_add_(1, ids, u * case["scale"])
        dl = ds * s * (1.0 - s) if case["scoring"] == "sigmoid" else s * (ds - (ds * s).sum(-1, keepdim=True))
        return dl.to(st["logits"].dtype)
    if op == "lora":
        L, r, K = st["a"].shape
        here = (st["index"].unsqueeze(1) == torch.arange(L, device="cuda")).float() * st["scale"]
        v = (st["x"].float() @ st["a"].float().view(L * r, K).t()).view(-1, L, r) * here.unsqueeze(-1)
        y = v.view(-1, L * r) @ st["b"].float().permute(0, 2, 1).reshape(L * r, -1)
        return (y + st["add"].float()).to(torch.bfloat16)
    dtype = getattr(torch, case["dtype"])
    if op == "dispatch":
        x, k = st["x"], case["topk"]
        offsets, slots, position = _order(st["ids"], case["E"], case["block"], _capacity(case))
        rows = torch.where((slots >= 0).unsqueeze(-1), x[(slots.clamp_min(0) // k).long()],
                           torch.zeros((), dtype=dtype, device="cuda"))
        return rows, offsets, slots, position
    offsets, slots, position = st["order"]
    if op == "dispatch_grad":
        return _rows_of(st["dout"], position).sum(1).to(dtype)
    if op == "combine":
        y = (_rows_of(st["y"], position) * st["w"].unsqueeze(-1)).sum(1)
        if st["add"] is not None:
            y = y + st["add"].float()
        return y.to(dtype)
    k = case["topk"]
    at = slots.clamp_min(0).long()
    g = st["g"].float()
    dy = torch.where((slots >= 0).unsqueeze(-1), st["w"].view(-1)[at].unsqueeze(-1) * g[at // k],
                     torch.zeros((), device="cuda"))
    dw = (_rows_of(st["y"], position) * g.unsqueeze(1)).sum(-1)
    return dy.to(dtype), dw


def _run_own(st):
    from int4_weight_only_moe_gb300 import dispatch, lora, routing
    case = st["case"]
    op = case["op"]
    if op == "route_grad":
        return routing.route_scored_backward(st["g"], st["logits"], st["ids"], scoring=case["scoring"],
                                             renormalize=case["renorm"], scale=case["scale"], out=st["out"])
    if op == "lora":
        return lora.apply(st["x"], st["a"], st["b"], st["index"], scale=st["scale"], add=st["add"], out=st["out"])
    order = dispatch.Order(*st["order"])
    if op == "dispatch":
        rows, order = dispatch.sort_gather(st["x"], st["ids"], case["E"], block=case["block"], out=st["out"], order=order)
        return rows, order.offsets, order.slots, order.position
    if op == "dispatch_grad":
        return dispatch.gather_backward(st["dout"], order, out=st["out"])
    if op == "combine":
        return dispatch.combine(st["y"], st["w"], order, add=st["add"], out=st["out"])
    return dispatch.combine_backward(st["g"], st["y"], st["w"], order, dy=st["out"][0], dweights=st["out"][1])


# ------------------------------------------------------------------- 64-bit definition


def exact(case, seed):
    st = prepare(case, seed)
    op, M = case["op"], case["M"]
    if op == "route_grad":
        l, ids, g = st["logits"].double(), st["ids"].long(), st["g"].double()
        s = torch.sigmoid(l) if case["scoring"] == "sigmoid" else torch.softmax(l, 1)
        p = torch.gather(s, 1, ids)
        # the Jacobian of the weights in the chosen scores, then of the scores in the logits
        eye = torch.eye(case["topk"], dtype=torch.float64, device="cuda").unsqueeze(0)
        if case["renorm"]:
            total = p.sum(1)[:, None, None]
            jac = eye / total - p.unsqueeze(2) / total ** 2
        else:
            jac = eye.expand(M, -1, -1)
        u = case["scale"] * torch.einsum("mi,mij->mj", g, jac)
        if case["scoring"] == "sigmoid":
            dl = torch.zeros_like(l)
            return dl.scatter_add(1, ids, u * p * torch.sigmoid(-torch.gather(l, 1, ids)))
        dl = -s * torch.einsum("mj,mj->m", u, p).unsqueeze(1)
        return dl.scatter_add(1, ids, u * p)
    if op == "lora":
        out = st["add"].double()
        for i in range(case["L"]):
            m = (st["index"] == i).nonzero().view(-1)
            v = torch.einsum("mk,rk->mr", st["x"][m].double(), st["a"][i].double())
            out[m] += st["scale"][i].double() * torch.einsum("mr,nr->mn", v, st["b"][i].double())
        return out
    E, k, block, capacity = case["E"], case["topk"], case["block"], _capacity(case)
    # an expert's slots counted along the list of slots, instead of a sort
    flat = st["ids"].view(-1).long()
    seen = torch.cumsum((flat.unsqueeze(1) == torch.arange(E, device="cuda")).int(), 0)
    ends = torch.cumsum((seen[-1] + block - 1).div(block, rounding_mode="floor") * block, 0)
    begins = torch.cat([ends.new_zeros(1), ends])
    known = flat >= 0
    e = flat.clamp_min(0)
    row = torch.where(known, begins[e] + seen.gather(1, e.unsqueeze(1)).squeeze(1) - 1, -1)
    del seen
    if op == "dispatch":
        slots = torch.full((capacity,), -1, dtype=torch.int32, device="cuda")
        slots[row[known]] = torch.arange(M * k, dtype=torch.int32, device="cuda")[known]
        rows = torch.zeros(capacity, case["K"], dtype=torch.float64, device="cuda")
        rows[row[known]] = st["x"].double().repeat_interleave(k, 0)[known]
        return rows, begins.to(torch.int32), slots, row.to(torch.int32).view(M, k)
    if op in ("dispatch_grad", "combine"):
        src = st["dout"] if op == "dispatch_grad" else st["y"]
        out = torch.zeros(M, case["K"], dtype=torch.float64, device="cuda")
        for j in range(k):
            r = row.view(M, k)[:, j]
            part = src[r.clamp_min(0)].double() * (r >= 0).unsqueeze(1)
            out += part if op == "dispatch_grad" else part * st["w"][:, j:j + 1].double()
        return out if op == "dispatch_grad" or st["add"] is None else out + st["add"].double()
    g = st["g"].double()
    dy = torch.zeros(capacity, case["K"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(M, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        r = row.view(M, k)[:, j]
        t = (r >= 0).nonzero().view(-1)
        dy[r[t]] = st["w"][t, j:j + 1].double() * g[t]
        dw[t, j] = torch.einsum("mk,mk->m", g[t], st["y"][r[t]].double())
    return dy, dw
