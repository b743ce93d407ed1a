"""Plain 64-bit definitions of the operators between the router and the experts (order of
the experts' rows, gather, combine, their gradients, the router's gradient) and of the
low-rank adapters, slot by slot, for the tests. Where a result is a sum, ``*_size`` gives
the sum of its terms' magnitudes, in whose units the tests' tolerances count roundings."""
import numpy as np


def order(ids, E, block=1, begin=0):
    """(offsets [E + 1], slots [rows], position [M, topk])."""
    M, topk = ids.shape
    n = M * topk
    cap = n + min(E, n) * (block - 1)
    offsets, slots, position = np.zeros(E + 1, np.int32), np.full(cap, -1, np.int32), np.full((M, topk), -1, np.int32)
    row = 0
    flat = ids.reshape(-1).astype(np.int64)
    for e in range(E):
        offsets[e] = row
        for i in np.nonzero(flat == begin + e)[0]:
            slots[row], position[i // topk, i % topk] = i, row
            row += 1
        row = -(-row // block) * block
    offsets[E] = row
    return offsets, slots, position


def gather(x, offsets, slots, topk, out):
    """``out`` with the rows of ``x`` in their places."""
    out = out.copy()
    for r in range(offsets[-1]):
        out[r] = x[slots[r] // topk] if slots[r] >= 0 else 0
    return out


def combine(y, w, position, add=None):
    M, topk = position.shape
    out = np.zeros((M, y.shape[1])) if add is None else add.astype(np.float64).copy()
    for t in range(M):
        for j in range(topk):
            if position[t, j] >= 0:
                out[t] += y[position[t, j]].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
    return out


def combine_size(y, w, position, add=None):
    return combine(np.abs(y), None if w is None else np.abs(w), position, None if add is None else np.abs(add))


def combine_backward(g, y, w, offsets, slots, position, dy):
    M, topk = position.shape
    dy, dw, size = dy.astype(np.float64).copy(), np.zeros((M, topk)), np.zeros((M, topk))
    dy[:offsets[-1]] = 0
    for t in range(M):
        for j in range(topk):
            r = position[t, j]
            if r >= 0:
                dy[r] = float(w[t, j]) * g[t].astype(np.float64)
                p = g[t].astype(np.float64) * y[r].astype(np.float64)
                dw[t, j], size[t, j] = p.sum(), np.abs(p).sum()
    return dy, dw, size


def route_weights(l, ids, scoring, renormalize, scale):
    """The router's weights of the chosen ``ids``, in 64 bits."""
    l = _clean(l)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    else:
        top = l.max(1, keepdims=True)
        e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
        s = e / np.maximum(e.sum(1, keepdims=True), 1e-300)
    ok = (ids >= 0) & (ids < l.shape[1])
    w = np.where(ok, np.take_along_axis(s, np.where(ok, ids, 0).astype(np.int64), 1), 0.0)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return w * scale


def _clean(l):
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    return np.minimum(l, float(np.finfo(np.float32).max))


def route_backward(g, l, ids, scoring, renormalize, scale):
    """(dlogits, size of the terms that make it up)."""
    M, E = l.shape
    topk = ids.shape[1]
    l = _clean(l)
    d, size = np.zeros((M, E)), np.zeros((M, E))
    for t in range(M):
        live = [j for j in range(topk) if 0 <= ids[t, j] < E and l[t, ids[t, j]] != -np.inf]
        at = [int(ids[t, j]) for j in live]
        gt = g[t, live].astype(np.float64)
        if not live:
            continue
        if scoring == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-np.maximum(l[t], -700.0)))
            s = np.where(l[t] == -np.inf, 0.0, s)
            rest = 1.0 / (1.0 + np.exp(np.clip(l[t], -700.0, 700.0)))
        else:
            s = np.exp(l[t] - max(l[t]))
            s = s / s.sum()
            if renormalize:  # the chosen alone, as they are
                s = np.exp(l[t] - max(l[t, at]))
            rest = np.ones(E)
        p = s[at]
        if renormalize:
            q = p / p.sum() if p.sum() > 0 else p * 0
            u_s, u_size = scale * q * (gt - (gt * q).sum()), abs(scale) * q * (np.abs(gt) + (np.abs(gt) * q).sum())
        else:
            u_s, u_size = scale * gt * p, abs(scale) * np.abs(gt) * p
        for i, e in enumerate(at):
            d[t, e] += u_s[i] * rest[e]
            size[t, e] += u_size[i] * rest[e]
        if scoring == "softmax" and not renormalize:
            d[t] -= s * u_s.sum()
            size[t] += s * u_size.sum()
    return d, size


def lora(x, a, b, index, scale=None, add=None):
    """(out, size of the second product's terms, size of both products' terms)."""
    M, (L, N) = len(x), b.shape[:2]
    out = np.zeros((M, N)) if add is None else add.astype(np.float64).copy()
    second, both = np.zeros((M, N)), np.zeros((M, N))
    for m in range(M):
        l = index[m]
        if 0 <= l < L:
            f = 1.0 if scale is None else float(scale[l])
            A, B, xm = a[l].astype(np.float64), b[l].astype(np.float64), x[m].astype(np.float64)
            v = A @ xm
            out[m] += f * (B @ v)
            second[m] = abs(f) * (np.abs(B) @ np.abs(v))
            both[m] = abs(f) * (np.abs(B) @ (np.abs(A) @ np.abs(xm)))
    return out, second, both
