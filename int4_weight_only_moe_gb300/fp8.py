"""8-bit block-scaled operators: quantisers, the matrix product, and the shared expert
that chains them (definitions: the ``moe_w4a16_fp8_*`` and ``moe_w4a16_shared_expert``
calls in ``include/moe_w4a16.h``).

Values are e4m3 (``torch.float8_e4m3fn``, or their bytes as ``torch.uint8``); a scale
belongs to 128 consecutive values of a row (activations, ``[M, ceil(K / 128)]``) or to a
block of 128 x 128 (weights, ``[ceil(N / 128), ceil(K / 128)]``).
"""
from __future__ import annotations

import functools

import torch

from . import BF16, F32, _check, _need, _new, lib, moe_w4a16_fp8_status, moe_w4a16_shared_expert_workspace_size
from .routing import _dense, _device, _handle, _on, _rows

BLOCK = 128
_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_BYTES = ("float8_e4m3fn", "uint8")
_E4M3 = {torch.float8_e4m3fn: 0, torch.uint8: 0}


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


def _bytes(t, shape, name, dev):
    """Address of a contiguous tensor of e4m3 values (or their bytes) of this shape on
    device ``dev``."""
    if t.dtype not in _E4M3 or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _need(t, _BYTES, shape, name)
        _on(t, dev, name)
    return t.data_ptr()


def _quantize(call, x, name, parts, rows_to_a_scale, q, s, stream):
    M, width, stride = _rows(x, name, _FLOATS)
    dev = _device(x, name)
    cols = width // parts
    scales = (M if rows_to_a_scale == 1 else _blocks(M), _blocks(cols))
    if q is None:
        q = _new((M, cols), torch.float8_e4m3fn, x.device, stream)
    if s is None:
        s = _new(scales, torch.float32, x.device, stream)
    _check(call(x.data_ptr(), _FLOATS[x.dtype], stride, M, cols, _bytes(q, (M, cols), "q", dev),
                _dense(s, torch.float32, scales, "s", dev), _handle(stream, dev)))
    return q, s


def quantize(x, q=None, s=None, stream=None):
    """``x`` [M, K] (bf16 or fp32) to ``(q e4m3 [M, K], s fp32 [M, ceil(K / 128)])``."""
    return _quantize(lib().moe_w4a16_fp8_quantize, x, "x", 1, 1, q, s, stream)


def swiglu_quantize(gate_up, q=None, s=None, stream=None):
    """SiLU(gate) * up of rows ``[gate | up]`` [M, 2 N], quantised: ``(q [M, N], s)``."""
    if gate_up.shape[-1] % 2:
        raise ValueError(f"gate_up: {gate_up.shape[-1]} columns, expected an even number")
    return _quantize(lib().moe_w4a16_fp8_swiglu_quantize, gate_up, "gate_up", 2, 1, q, s, stream)


def quantize_weight(w, q=None, s=None, stream=None):
    """A weight [N, K] to ``(q e4m3 [N, K], s fp32 [ceil(N / 128), ceil(K / 128)])``."""
    return _quantize(lib().moe_w4a16_fp8_quantize_weight, w, "w", 1, BLOCK, q, s, stream)


def matmul(a, a_s, b, b_s, add=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """``(a a_s) (b b_s)^T`` (+ ``add``) of 8-bit ``a`` [M, K] and ``b`` [N, K]: [M, N] in
    ``out_dtype`` (bf16 or fp32; that of ``out`` where it is given)."""
    M, K, lda = _rows(a, "a", _E4M3)
    N, b_cols, ldb = _rows(b, "b", _E4M3)
    dev = _device(a, "a")
    _on(b, dev, "b")
    if b_cols != K:
        raise ValueError(f"b: shape {tuple(b.shape)}, expected {K} columns")
    sa = _dense(a_s, torch.float32, (M, _blocks(K)), "a_s", dev)
    sb = _dense(b_s, torch.float32, (_blocks(N), _blocks(K)), "b_s", dev)
    plus = 0 if add is None else _dense(add, torch.bfloat16, (M, N), "add", dev)
    if out is None:
        out = _new((M, N), out_dtype, a.device, stream)
    if out.dtype not in _FLOATS:
        raise ValueError(f"out: dtype {out.dtype}, expected one of {tuple(_FLOATS)}")
    _check(lib().moe_w4a16_fp8_matmul(
        a.data_ptr(), lda, sa, b.data_ptr(), ldb, sb, plus, _dense(out, out.dtype, (M, N), "out", dev), _FLOATS[out.dtype],
        M, N, K, _handle(stream, dev)))
    return out


_POOL_BYTES = 16 << 20
_workspace_size = functools.lru_cache(maxsize=256)(moe_w4a16_shared_expert_workspace_size)


def shared_expert(hidden, w1, w1_s, w2, w2_s, add=None, out=None, workspace=None, stream=None):
    """The shared expert's feed-forward of ``hidden`` bf16 [M, K] (+ ``add`` bf16 [M, K], the
    routed experts' output): bf16 [M, K].

    ``w1`` [2 N, K] holds the gate rows, then the up rows, ``w2`` [K, N] the down
    projection. ``workspace``: uint8, of
    ``moe_w4a16_shared_expert_workspace_size(M, K, N)`` bytes; where it is not given, up to
    16 MiB come from the library's stream-ordered pool (a third of the time of a tensor's
    allocation, which a small batch's call would wait for), more from torch.
    """
    M, K = shape = hidden.shape
    N = w2.shape[1]
    dev = _device(hidden, "hidden")
    x = _dense(hidden, torch.bfloat16, (M, K), "hidden", dev)
    kb, nb = _blocks(K), _blocks(N)
    weights = (_bytes(w1, (2 * N, K), "w1", dev), _dense(w1_s, torch.float32, (_blocks(2 * N), kb), "w1_s", dev),
               _bytes(w2, (K, N), "w2", dev), _dense(w2_s, torch.float32, (kb, nb), "w2_s", dev))
    plus = 0 if add is None else _dense(add, torch.bfloat16, shape, "add", dev)
    if out is None:
        out = _new(shape, torch.bfloat16, hidden.device, stream)
    y = _dense(out, torch.bfloat16, shape, "out", dev)
    if workspace is None and (need := _workspace_size(M, K, N)) > _POOL_BYTES:
        workspace = _new((need,), torch.uint8, hidden.device, stream)
    ws = size = 0
    if workspace is not None:
        _on(workspace, dev, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, size = workspace.data_ptr(), workspace.nbytes
    _check(lib().moe_w4a16_shared_expert(x, *weights, plus, y, M, K, N, ws, size, _handle(stream, dev)))
    return out


def status(stream=None) -> int:
    """Status of the products on the current device since the last call (0: clean);
    synchronises ``stream``."""
    return moe_w4a16_fp8_status(stream)
