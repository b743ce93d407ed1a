"""8-bit block-scaled operators: quantisers, the matrix product, and the shared expert
that chains them (definitions: the ``moe_w4a16_fp8_*`` and ``moe_w4a16_shared_expert``
calls in ``include/moe_w4a16.h``).

Values are e4m3 (``torch.float8_e4m3fn``, or their bytes as ``torch.uint8``); a scale
belongs to 128 consecutive values of a row (activations, ``[M, ceil(K / 128)]``) or to a
block of 128 x 128 (weights, ``[ceil(N / 128), ceil(K / 128)]``).
"""
from __future__ import annotations

import torch

from . import (BF16, F32, _need, moe_w4a16_fp8_matmul, moe_w4a16_fp8_quantize, moe_w4a16_fp8_quantize_weight,
               moe_w4a16_fp8_swiglu_quantize, moe_w4a16_shared_expert, moe_w4a16_shared_expert_workspace_size)
from .routing import _lend, _rows

BLOCK = 128
_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_BYTES = ("float8_e4m3fn", "uint8")
_E4M3 = {torch.float8_e4m3fn: 0, torch.uint8: 0}


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _quantize(call, x, name, cols, scale_rows, q, s, stream):
    stride = _rows(x, name, _FLOATS)
    M = x.shape[0]
    if q is None:
        q = torch.empty((M, cols), dtype=torch.float8_e4m3fn, device=x.device)
        _lend(stream, q)
    else:
        _need(q, _BYTES, (M, cols), "q")
    if s is None:
        s = torch.empty((scale_rows, _blocks(cols)), dtype=torch.float32, device=x.device)
        _lend(stream, s)
    else:
        _need(s, ("float32",), (scale_rows, _blocks(cols)), "s")
    call(x, _FLOATS[x.dtype], stride, M, cols, q, s, stream)
    return q, s


def quantize(x, q=None, s=None, stream=None):
    """``x`` [M, K] (bf16 or fp32) to ``(q e4m3 [M, K], s fp32 [M, ceil(K / 128)])``."""
    return _quantize(moe_w4a16_fp8_quantize, x, "x", x.shape[-1], x.shape[0], q, s, stream)


def swiglu_quantize(gate_up, q=None, s=None, stream=None):
    """SiLU(gate) * up of rows ``[gate | up]`` [M, 2 N], quantised: ``(q [M, N], s)``."""
    if gate_up.shape[-1] % 2:
        raise ValueError(f"gate_up: {gate_up.shape[-1]} columns, expected an even number")
    return _quantize(moe_w4a16_fp8_swiglu_quantize, gate_up, "gate_up", gate_up.shape[-1] // 2, gate_up.shape[0],
                     q, s, stream)


def quantize_weight(w, q=None, s=None, stream=None):
    """A weight [N, K] to ``(q e4m3 [N, K], s fp32 [ceil(N / 128), ceil(K / 128)])``."""
    return _quantize(moe_w4a16_fp8_quantize_weight, w, "w", w.shape[-1], _blocks(w.shape[0]), q, s, stream)


def matmul(a, a_s, b, b_s, add=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """``(a a_s) (b b_s)^T`` (+ ``add``) of 8-bit ``a`` [M, K] and ``b`` [N, K]: [M, N] in
    ``out_dtype`` (bf16 or fp32; that of ``out`` where it is given)."""
    lda, ldb = _rows(a, "a", _E4M3), _rows(b, "b", _E4M3)
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError(f"b: shape {tuple(b.shape)}, expected {K} columns")
    _need(a_s, ("float32",), (M, _blocks(K)), "a_s")
    _need(b_s, ("float32",), (_blocks(N), _blocks(K)), "b_s")
    if add is not None:
        _need(add, ("bfloat16",), (M, N), "add")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=a.device)
        _lend(stream, out)
    else:
        _need(out, ("bfloat16", "float32"), (M, N), "out")
    if out.dtype not in _FLOATS:
        raise ValueError(f"out_dtype: {out.dtype}, expected one of {tuple(_FLOATS)}")
    moe_w4a16_fp8_matmul(a, lda, a_s, b, ldb, b_s, add, out, _FLOATS[out.dtype], M, N, K, stream)
    return out


def shared_expert(hidden, w1, w1_s, w2, w2_s, add=None, out=None, workspace=None, stream=None):
    """The shared expert's feed-forward of ``hidden`` bf16 [M, K] (+ ``add`` bf16 [M, K], the
    routed experts' output): bf16 [M, K].

    ``w1`` [2 N, K] holds the gate rows, then the up rows, ``w2`` [K, N] the down
    projection. ``workspace`` (uint8, of
    ``moe_w4a16_shared_expert_workspace_size(M, K, N)`` bytes) is allocated where it is not
    given.
    """
    M, K = hidden.shape
    N = w2.shape[1]
    _need(hidden, ("bfloat16",), (M, K), "hidden")
    _need(w1, _BYTES, (2 * N, K), "w1")
    _need(w1_s, ("float32",), (_blocks(2 * N), _blocks(K)), "w1_s")
    _need(w2, _BYTES, (K, N), "w2")
    _need(w2_s, ("float32",), (_blocks(K), _blocks(N)), "w2_s")
    if add is not None:
        _need(add, ("bfloat16",), (M, K), "add")
    if out is None:
        out = torch.empty((M, K), dtype=torch.bfloat16, device=hidden.device)
        _lend(stream, out)
    else:
        _need(out, ("bfloat16",), (M, K), "out")
    if workspace is None:
        need = moe_w4a16_shared_expert_workspace_size(M, K, N)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=hidden.device)
        _lend(stream, workspace)
    moe_w4a16_shared_expert(hidden, w1, w1_s, w2, w2_s, add, out, M, K, N, workspace, stream)
    return out
