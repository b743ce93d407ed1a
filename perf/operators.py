"""Measured cases of the operators around the routed experts: the scored router, the
8-bit block quantiser, the 8-bit block-scaled matrix product, and the shared expert
that chains the last two.

``run`` computes each in elementary torch operations (fp32, rounded once at the end)
or, where ``own`` is true, with the library's kernels. Definitions:

* route    s = sigmoid(l) or softmax(l); c = s + bias; with groups, a group counts the
           sum of its ``group_top`` largest c and only the ``topk_group`` best groups
           stay; the ids are the ``topk`` largest c (equal ones: lowest id first), the
           weights s of those, divided by their sum if ``renorm``, times ``scale``.
* quantize per row and 128 columns: s = max(max|x| / 448, 2^-126), q = e4m3(x / s), the
           scale and the quotient 32-bit numbers.
           "swiglu": x = g / (1 + exp(-g)) * u of a row [g | u].
* matmul   out[m, n] = sum_k a[m, k] as[m, k/128] b[n, k] bs[n/128, k/128] (+ add[m, n]).
* shared   quantize -> matmul with [gate; up] -> swiglu quantize -> matmul with down
           (+ add), the products' sums unrounded in between.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # one token of a decode step through the layer of this framework's benchmark
        # (384 experts, top-8), sigmoid scores with a balance bias
        dict(name="route_decode", op="route", M=1, E=384, topk=8, scoring="sigmoid", bias=True, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=2.5, dtype="float32"),
        # a ragged verify batch over 8 groups of 32 experts, 4 groups a token, bf16 gate output
        dict(name="route_grouped", op="route", M=333, E=256, topk=8, scoring="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, renorm=True, scale=2.5, dtype="bfloat16"),
        # a prompt of 16,384 tokens
        dict(name="route_prompt", op="route", M=16384, E=384, topk=8, scoring="sigmoid", bias=True, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=2.5, dtype="float32"),
        # softmax scores limited to 3 of 8 groups of 20, weights as they are; odd token count
        dict(name="route_softmax", op="route", M=4097, E=160, topk=6, scoring="softmax", bias=False, n_group=8,
             topk_group=3, group_top=1, renorm=False, scale=16.0, dtype="float32"),
        # the hidden states of a small decode batch, before the gate/up product
        dict(name="quant_batch", op="quantize", M=17, N=7168, swiglu=False),
        # the gate/up outputs of a prompt, before the down product
        dict(name="quant_swiglu", op="quantize", M=8191, N=2048, swiglu=True),
        # gate/up product of one token: weight streaming
        dict(name="mm_decode", op="matmul", M=1, N=4096, K=7168, out="bfloat16", add=False),
        # down product of a verify batch, added to the routed experts' output
        dict(name="mm_verify", op="matmul", M=90, N=7168, K=2048, out="bfloat16", add=True),
        # gate/up product of a prompt: tensor-core bound
        dict(name="mm_prompt", op="matmul", M=8192, N=4096, K=7168, out="bfloat16", add=False),
        # ragged everywhere (a last block of 16 along K, a last block of 104 along N), fp32 output
        dict(name="mm_ragged", op="matmul", M=777, N=1000, K=1936, out="float32", add=False),
        # the whole shared expert: a decode batch, and a prompt chunk
        dict(name="shared_decode", op="shared", M=4, K=7168, N=2048, add=True),
        dict(name="shared_prompt", op="shared", M=2048, K=7168, N=2048, add=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "route", "quantize", "matmul", "matmul", "shared"])
    if op == "route":
        n_group = rng.choice([1, 1, 2, 4, 8, 16])
        size = _log_int(rng, max(2, 16 // n_group), 384 // n_group)
        E = n_group * size
        topk_group = rng.randint(1, n_group)
        topk = rng.randint(1, min(topk_group * size, 12))
        scoring = rng.choice(["sigmoid", "sigmoid", "softmax"])
        bias = scoring == "sigmoid" and rng.random() < 0.8
        return dict(op=op, M=_log_int(rng, 1, 16384), E=E, topk=topk, scoring=scoring, bias=bias, n_group=n_group,
                    topk_group=topk_group, group_top=2 if bias else 1, renorm=rng.random() < 0.7,
                    scale=rng.choice([1.0, 2.5, 16.0]), dtype=rng.choice(["float32", "bfloat16"]))
    if op == "quantize":
        swiglu = rng.random() < 0.5
        return dict(op=op, M=_log_int(rng, 1, 8192), N=16 * _log_int(rng, 4, 128 if swiglu else 448), swiglu=swiglu)
    if op == "matmul":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 64, 4096), K=16 * _log_int(rng, 8, 448),
                    out=rng.choice(["bfloat16", "bfloat16", "float32"]), add=rng.random() < 0.4)
    return dict(op=op, M=_log_int(rng, 1, 2048), K=128 * _log_int(rng, 4, 56), N=128 * _log_int(rng, 2, 16),
                add=rng.random() < 0.5)


def work(case):
    M = case["M"]
    up = lambda n: -(-n // 128)  # noqa: E731
    if case["op"] == "route":
        E, k = case["E"], case["topk"]
        item = 4 if case["dtype"] == "float32" else 2
        return {"bytes": M * E * item + (4 * E if case["bias"] else 0) + 8 * M * k, "flops": 0}
    if case["op"] == "quantize":
        N = case["N"]
        return {"bytes": M * N * 2 * (2 if case["swiglu"] else 1) + M * N + 4 * M * up(N), "flops": 0}
    if case["op"] == "matmul":
        N, K = case["N"], case["K"]
        out = 2 if case["out"] == "bfloat16" else 4
        return {"bytes": M * K + N * K + 4 * up(K) * (M + up(N)) + M * N * out + (2 * M * N if case["add"] else 0),
                "flops": 2 * M * N * K}
    N, K = case["N"], case["K"]
    return {"bytes": 3 * N * K + 4 * 3 * up(N) * up(K) + M * K * (6 if case["add"] else 4), "flops": 6 * M * N * K}


# ----------------------------------------------------------------------------- inputs


def _scores64(l, scoring):
    l = l.double()
    return torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, -1)


def _undecided(l, bias, case):
    """Rows whose selection hangs on less than the rounding of 32 bits: two values that it
    compares are neither equal nor apart. Whole numbers have to be equal, so prepare
    draws such rows again."""
    c = _scores64(l, case["scoring"])
    if bias is not None:
        c = c + bias.double()
    M, E = c.shape
    G, k = case["n_group"], case["topk"]

    def near(a, b):
        d = a - b
        return (d != 0) & (d < 4e-6 * torch.maximum(a.abs(), torch.full_like(a, 0.5 if bias is not None else 0.0)))

    bad = torch.zeros(M, dtype=torch.bool, device=l.device)
    if G > 1:
        g = c.view(M, G, E // G).sort(dim=-1, descending=True)[0][..., :case["group_top"]].sum(-1)
        order = g.sort(dim=-1, descending=True, stable=True)
        t = case["topk_group"]
        if t < G:
            bad |= near(order[0][:, t - 1], order[0][:, t])
        keep = torch.zeros(M, G, dtype=torch.bool, device=l.device).scatter_(1, order[1][:, :t], True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -1e30))
    v = c.sort(dim=-1, descending=True)[0][:, :k + 1]
    bad |= near(v[:, :-1], v[:, 1:]).any(-1)
    return bad


def _blocks_amax(w):
    """max |w| of every 128 x 128 block of [N, K] (ragged at the ends)."""
    N, K = w.shape
    p = torch.nn.functional.pad(w.abs(), (0, -K % 128, 0, -N % 128))
    return p.view(-(-N // 128), 128, -(-K // 128), 128).amax((1, 3))


def _scale_of(amax):
    # (a quotient of tensors: dividing by a Python number multiplies by its rounded inverse)
    return (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(TINY)


def _weight(gen, N, K):
    """8-bit weights [N, K] and their scales, one for each 128 x 128 block."""
    w = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    s = _scale_of(_blocks_amax(w))
    q = (w / _spread(s, N, K)).to(torch.float8_e4m3fn)
    return q, s


def _spread(s, N, K):
    return s.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]


def _hidden(gen, M, K):
    """Hidden states: normal, a few channels several times the rest."""
    x = torch.randn(M, K, generator=gen, device="cuda")
    gain = torch.ones(K, device="cuda")
    gain[torch.randint(0, K, (max(1, K // 200),), generator=gen, device="cuda")] = 8.0
    return (x * gain).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    M = case["M"]
    st = dict(case=dict(case))
    up = lambda n: -(-n // 128)  # noqa: E731
    new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if case["op"] == "route":
        E, k = case["E"], case["topk"]
        dtype = getattr(torch, case["dtype"])
        st["bias"] = torch.randn(E, generator=gen, device="cuda") * 0.05 if case["bias"] else None
        l = (torch.randn(M, E, generator=gen, device="cuda") * 1.5).to(dtype)
        for _ in range(20):
            bad = _undecided(l, st["bias"], case).nonzero().view(-1)
            if not bad.numel():
                break
            l[bad] = (torch.randn(bad.numel(), E, generator=gen, device="cuda") * 1.5).to(dtype)
        st["logits"] = l
        st["out"] = (new(M, k, dtype=torch.int32), new(M, k, dtype=torch.float32))
    elif case["op"] == "quantize":
        N = case["N"]
        if case["swiglu"]:
            st["x"] = (torch.randn(M, 2 * N, generator=gen, device="cuda") * 2.0).to(torch.bfloat16)
        else:
            st["x"] = _hidden(gen, M, N)
        st["out"] = (new(M, N, dtype=torch.float8_e4m3fn), new(M, up(N), dtype=torch.float32))
    elif case["op"] == "matmul":
        N, K = case["N"], case["K"]
        st["a"], st["a_s"] = _quantize(_hidden(gen, M, K).float())
        st["b"], st["b_s"] = _weight(gen, N, K)
        st["add"] = torch.randn(M, N, generator=gen, device="cuda").to(torch.bfloat16) if case["add"] else None
        st["out"] = new(M, N, dtype=getattr(torch, case["out"]))
    else:
        N, K = case["N"], case["K"]
        st["x"] = _hidden(gen, M, K)
        st["w1"], st["w1_s"] = _weight(gen, 2 * N, K)
        st["w2"], st["w2_s"] = _weight(gen, K, N)
        st["add"] = torch.randn(M, K, generator=gen, device="cuda").to(torch.bfloat16) if case["add"] else None
        st["out"] = new(M, K, dtype=torch.bfloat16)
    return st


# ------------------------------------------------------------------------------- runs


def _rows_blocks(x):
    """[M, K] -> [M, ceil(K / 128), 128], zeros behind the end."""
    M, K = x.shape
    if K % 128:
        x = torch.nn.functional.pad(x, (0, -K % 128))
    return x.view(M, -1, 128)


def _quantize(x):
    M, K = x.shape
    b = _rows_blocks(x)
    s = _scale_of(b.abs().amax(-1))
    q = (b / s[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(M, -1)[:, :K].contiguous(), s


def _swiglu(x):
    N = x.shape[1] // 2
    g, u = x[:, :N], x[:, N:]
    return g / (1.0 + torch.exp(-g)) * u


def _matmul(a, a_s, b, b_s):
    M, K = a.shape
    fa = a.float() * a_s.repeat_interleave(128, 1)[:, :K]
    fb = b.float() * _spread(b_s, b.shape[0], K)
    return fa @ fb.t()


def _route(l, bias, case):
    l = l.float()
    if case["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    c = s if bias is None else s + bias
    M, E = c.shape
    G = case["n_group"]
    if G > 1:
        g = c.view(M, G, E // G).sort(dim=-1, descending=True)[0][..., :case["group_top"]].sum(-1)
        top = g.sort(dim=-1, descending=True, stable=True)[1][:, :case["topk_group"]]
        keep = torch.zeros(M, G, dtype=torch.bool, device=c.device).scatter_(1, top, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, torch.full_like(c, -math.inf))
    ids = c.sort(dim=-1, descending=True, stable=True)[1][:, :case["topk"]]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), w * case["scale"]


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "route":
        return _route(st["logits"], st["bias"], case)
    if op == "quantize":
        x = st["x"].float()
        return _quantize(_swiglu(x) if case["swiglu"] else x)
    if op == "matmul":
        y = _matmul(st["a"], st["a_s"], st["b"], st["b_s"])
        if st["add"] is not None:
            y = y + st["add"]
        return y.to(getattr(torch, case["out"]))
    h = _swiglu(_matmul(*_quantize(st["x"].float()), st["w1"], st["w1_s"]))
    y = _matmul(*_quantize(h), st["w2"], st["w2_s"])
    if st["add"] is not None:
        y = y + st["add"]
    return y.to(torch.bfloat16)


def _run_own(st):
    from int4_weight_only_moe_gb300 import fp8, routing
    case = st["case"]
    op = case["op"]
    if op == "route":
        return routing.route_scored(st["logits"], case["topk"], scoring=case["scoring"], bias=st["bias"],
                                    n_group=case["n_group"], topk_group=case["topk_group"],
                                    group_top=case["group_top"], renormalize=case["renorm"], scale=case["scale"],
                                    ids=st["out"][0], weights=st["out"][1])
    if op == "quantize":
        call = fp8.swiglu_quantize if case["swiglu"] else fp8.quantize
        return call(st["x"], q=st["out"][0], s=st["out"][1])
    if op == "matmul":
        return fp8.matmul(st["a"], st["a_s"], st["b"], st["b_s"], add=st["add"], out=st["out"])
    return fp8.shared_expert(st["x"], st["w1"], st["w1_s"], st["w2"], st["w2_s"], add=st["add"], out=st["out"])


# ------------------------------------------------------------------- 64-bit definition


def _e4m3_64(v):
    """Nearest e4m3 value (4 significant bits, ties to even, smallest step 2^-9, at most 448)."""
    v = v.clamp(-E4M3_MAX, E4M3_MAX)
    _, e = torch.frexp(v)  # |v| in [2^(e-1), 2^e)
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(v / step) * step


def _quantize_64(x):
    M, K = x.shape
    nb = -(-K // 128)
    full = torch.zeros(M, nb * 128, dtype=torch.float64, device=x.device)
    full[:, :K] = x
    full = full.view(M, nb, 128)
    s = torch.maximum(full.abs().amax(2) / E4M3_MAX, torch.full((M, nb), TINY, dtype=torch.float64, device=x.device))
    # the scale is kept in 32 bits, and so is the quotient that is rounded to 8: with both
    # bf16, x / s often is the middle of two 8-bit values but for these roundings
    s = s.float().double()
    q = _e4m3_64((full / s.unsqueeze(2)).float().double())
    return q.reshape(M, nb * 128)[:, :K], s


def _dequant_64(q, s, rows):
    """q [R, K] times its scale: s [R, K/128] (rows = 1) or [R/128, K/128] (rows = 128)."""
    R, K = q.shape
    r = torch.arange(R, device=q.device) // rows
    k = torch.arange(K, device=q.device) // 128
    return q.double() * s.double()[r][:, k]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        s = _scores64(st["logits"], case["scoring"])
        c = s if st["bias"] is None else s + st["bias"].double()
        M, E = c.shape
        size = E // case["n_group"]
        if case["n_group"] > 1:
            best = torch.topk(c.view(M, -1, size), min(case["group_top"], size), dim=2).values.sum(2)
            t = case["topk_group"]
            # a group stays if fewer than t others come before it (equal ones by their number)
            ahead = best.unsqueeze(1) > best.unsqueeze(2)
            lower = torch.arange(best.shape[1], device=c.device)
            tie = (best.unsqueeze(1) == best.unsqueeze(2)) & (lower[None, None, :] < lower[None, :, None])
            stays = (ahead | tie).sum(2) < t
            c = c.masked_fill(~stays.unsqueeze(2).expand(M, case["n_group"], size).reshape(M, E), -math.inf)
        ids = []
        for _ in range(case["topk"]):  # argmax by argmax, the lowest id of equal ones
            top = c.amax(1, keepdim=True)
            i = torch.where(c == top, torch.arange(E, device=c.device), E).amin(1, keepdim=True)
            ids.append(i)
            c = c.scatter(1, i, -math.inf)
        ids = torch.cat(ids, 1)
        w = s.gather(1, ids)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return ids.to(torch.int32), w * case["scale"]
    if op == "quantize":
        x = st["x"].double()
        if case["swiglu"]:
            g, u = x.chunk(2, 1)
            x = g * torch.sigmoid(g) * u
        return _quantize_64(x)
    if op == "matmul":
        y = torch.einsum("mk,nk->mn", _dequant_64(st["a"], st["a_s"], 1), _dequant_64(st["b"], st["b_s"], 128))
        return y if st["add"] is None else y + st["add"].double()
    N = case["N"]
    q, s = _quantize_64(st["x"].double())
    gu = torch.einsum("mk,nk->mn", _dequant_64(q, s, 1), _dequant_64(st["w1"], st["w1_s"], 128))
    q, s = _quantize_64(gu[:, :N] * torch.sigmoid(gu[:, :N]) * gu[:, N:])
    y = torch.einsum("mk,nk->mn", _dequant_64(q, s, 1), _dequant_64(st["w2"], st["w2_s"], 128))
    return y if st["add"] is None else y + st["add"].double()
