"""Float64 numpy definitions of the operators around the routed experts: the scored
router, the 8-bit block quantisers and product, the shared expert. One function per
definition; shares no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -126


def e4m3_values(bits):
    """The values of e4m3 bytes (sign, 4 exponent bits of bias 7, 3 fraction bits; the
    pattern of all ones is NaN, there is no infinity)."""
    b = np.asarray(bits, dtype=np.uint8)
    sign = np.where(b & 0x80, -1.0, 1.0)
    e, m = ((b >> 3) & 15).astype(np.int64), (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * np.exp2((e - 7).astype(np.float64)))
    return np.where((b & 0x7F) == 0x7F, np.nan, sign * v)


def e4m3_round(v):
    """Nearest e4m3 value, ties to the even one, magnitudes above 448 to 448."""
    v = np.asarray(v, dtype=np.float64)
    grid = e4m3_values(np.arange(127, dtype=np.uint8))  # 0 .. 448 ascending, even bytes have even fractions
    a = np.minimum(np.abs(v), E4M3_MAX)
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    pick = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isnan(v), np.nan, np.copysign(grid[pick], v))


def _pad_blocks(x, axis):
    n = x.shape[axis]
    pad = [(0, 0)] * x.ndim
    pad[axis] = (0, -n % BLOCK)
    return np.pad(x, pad)


def _scales(amax):
    """32-bit scales max(amax / 448, 2^-126)."""
    return np.maximum((np.asarray(amax, np.float64) / E4M3_MAX), SCALE_FLOOR).astype(np.float32)


def _quotient(x, s):
    """x / s as the 32-bit number that is rounded to 8 bits."""
    return (np.asarray(x, np.float64) / np.asarray(s, np.float64)).astype(np.float32).astype(np.float64)


def quantize(x):
    """``x`` [M, K] to (e4m3 values float64 [M, K], scales float32 [M, ceil(K / 128)])."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    b = _pad_blocks(x, 1).reshape(M, -1, BLOCK)
    s = _scales(np.abs(b).max(-1, initial=0.0))
    return e4m3_round(_quotient(b, s[..., None])).reshape(M, -1)[:, :K], s


def quantize_weight(w):
    """``w`` [N, K] to (values [N, K], scales float32 [ceil(N / 128), ceil(K / 128)])."""
    w = np.asarray(w, np.float64)
    N, K = w.shape
    p = np.abs(_pad_blocks(_pad_blocks(w, 0), 1))
    s = _scales(p.reshape(-(-N // BLOCK), BLOCK, -(-K // BLOCK), BLOCK).max((1, 3)))
    return e4m3_round(_quotient(w, spread_weight_scales(s, N, K))), s


def spread_weight_scales(s, N, K):
    return np.repeat(np.repeat(np.asarray(s, np.float64), BLOCK, 0)[:N], BLOCK, 1)[:, :K]


def dequantize(q, s):
    return q * np.repeat(np.asarray(s, np.float64), BLOCK, 1)[:, :q.shape[1]]


def dequantize_weight(q, s):
    return q * spread_weight_scales(s, *q.shape)


def silu(z):
    z = np.asarray(z, np.float64)
    return z / (1.0 + np.exp(-z))


def matmul(a, a_s, b, b_s, add=None):
    """(values, absolute sums): sum of the products, and of their magnitudes (the measure
    of its rounding errors)."""
    fa, fb = dequantize(a, a_s), dequantize_weight(b, b_s)
    y = fa @ fb.T
    if add is not None:
        y = y + add
    return y, np.abs(fa) @ np.abs(fb).T


def shared_expert(x, w1, w1_s, w2, w2_s, add=None):
    N = w2.shape[1]
    gu, _ = matmul(*quantize(x), w1, w1_s)
    y, _ = matmul(*quantize(silu(gu[:, :N]) * gu[:, N:]), w2, w2_s)
    return y if add is None else y + add


def route_scored(logits, topk, scoring="sigmoid", bias=None, n_group=1, topk_group=1, group_top=1,
                 renormalize=True, scale=1.0):
    """(ids int64 [M, topk], weights [M, topk], margin [M]). ``margin`` is the smallest
    non-zero difference between two values that a row's selection compares at its border,
    as a share of the largest score and value there (inf where there is none): a row of
    smaller margin than the arithmetic's relative error may be selected either way."""
    l = np.asarray(logits, np.float64)
    M, E = l.shape
    masked = np.isnan(l) | (l == -np.inf)
    l = np.minimum(np.where(masked, -np.inf, l), np.finfo(np.float32).max)
    if scoring == "sigmoid":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-l))
    else:
        top = np.where(masked.all(1, keepdims=True), 0.0, l.max(1, keepdims=True))
        e = np.exp(l - top)
        z = e.sum(1, keepdims=True)
        s = e / np.where(z == 0, 1.0, z)
    c = s if bias is None else s + np.asarray(bias, np.float64)
    c = np.where(masked, -np.inf, c)
    size = E // n_group
    ids = np.zeros((M, topk), np.int64)
    w = np.zeros((M, topk))
    margin = np.full(M, np.inf)

    def near(row, values):
        v = np.asarray(values)
        v = v[np.isfinite(v)]
        d = v[:-1] - v[1:]
        if (d > 0).any():
            margin[row] = min(margin[row], d[d > 0].min() / max(np.abs(v).max(), s[row].max()))

    for t in range(M):
        groups = c[t].reshape(n_group, size)
        best = np.sort(groups, 1)[:, ::-1]
        value = best[:, 0].copy()
        if group_top == 2 and size > 1:
            value += np.where(np.isfinite(best[:, 1]), best[:, 1], 0.0)
        order = np.argsort(-value, kind="stable")
        if topk_group < n_group:
            near(t, value[order[topk_group - 1:topk_group + 1]])
        stay = np.zeros(n_group, bool)
        stay[order[:topk_group]] = True
        cand = np.flatnonzero(np.repeat(stay, size))
        pick = cand[np.argsort(-c[t, cand], kind="stable")]
        near(t, c[t, pick[:topk + 1]])
        ids[t] = pick[:topk]
        w[t] = s[t, ids[t]]
        if renormalize:
            total = w[t].sum()
            if total > 0:
                w[t] /= total
        w[t] *= scale
    return ids, w, margin
