"""Tokens sorted by expert and back, around expert products of the caller's own
(definitions: the ``moe_w4a16_dispatch_*`` and ``moe_w4a16_combine*`` calls in
``include/moe_w4a16.h``).

    rows, order = sort_gather(hidden, ids, E, block=128)   # ids: routing.route_scored
    y           = the experts' products of rows[order.offsets[e]:order.offsets[e + 1]]
    out         = combine(y, weights, order, add=shared)
    dy, dw      = combine_backward(dout, y, weights, order)
    dhidden     = gather_backward(drows, order)            # drows: the products' gradient
    dlogits     = routing.route_scored_backward(dw, logits, ids)
"""
from __future__ import annotations

import functools
from typing import NamedTuple

import torch

from . import BF16, E4M3, F32, _check, _new, lib, moe_w4a16_dispatch_rows
from .routing import _dense, _device, _fast, _handle, _rows

_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_MOVED = {**_FLOATS, torch.float8_e4m3fn: E4M3, torch.uint8: E4M3}

_order_rows = functools.lru_cache(maxsize=1024)(moe_w4a16_dispatch_rows)


class Order(NamedTuple):
    """The experts' rows: where each expert's begin (int32 [E + 1]), the slot t * topk + j of
    each row (int32 [rows], -1: none), the row of each slot (int32 [M, topk], -1: none)."""
    offsets: torch.Tensor
    slots: torch.Tensor
    position: torch.Tensor


def rows(M: int, topk: int, E: int, block: int = 1) -> int:
    """Rows that an order of these sizes has room for."""
    n = _order_rows(M, topk, E, block)
    if n < 0:
        raise ValueError(f"{M} tokens of {topk} choices, {E} experts in blocks of {block}: not supported")
    return n


@functools.lru_cache(maxsize=1024)
def _block_of(M, topk, E, cap):
    """The block of an order of ``cap`` rows; 0 where there is none."""
    n = M * topk
    block = 1 if not n or not E else (cap - n) // min(E, n) + 1
    return block if block > 0 and cap == _order_rows(M, topk, E, block) else 0


def _parts(order, dev):
    """(addresses of the order's tensors, M, topk, E, rows, block)"""
    offsets, slots, position = order
    try:
        (E,), (cap,), (M, topk) = offsets.shape, slots.shape, position.shape
    except ValueError:
        raise ValueError("order: expected offsets [E + 1], slots [rows] and position [M, topk]") from None
    E -= 1
    block = _block_of(M, topk, E, cap)
    if not block:
        raise ValueError(f"order: {cap} rows for {M} tokens of {topk} choices and {E} experts")
    at = (_int32(offsets, "order.offsets", dev), _int32(slots, "order.slots", dev), _int32(position, "order.position", dev))
    return at, M, topk, E, cap, block


def _int32(t, name, dev):
    """Address of a contiguous int32 tensor of any shape on device ``dev``."""
    if t.dtype is not torch.int32 or t.get_device() != dev or not t.is_contiguous():
        return _dense(t, torch.int32, t.shape, name, dev)
    return t.data_ptr()


def _matrix(t, name):
    """(rows, columns, device) of a contiguous bf16 or fp32 matrix on the current device."""
    if t.dtype not in _FLOATS or not t.is_contiguous() or t.dim() != 2:
        _rows(t, name, _FLOATS)
        raise ValueError(f"{name} must be contiguous")
    rows, cols = t.shape
    return rows, cols, _device(t, name)


def _order_for(topk_ids, E, block, expert_range, order, dev, stream):
    """(the order to write, addresses, M, topk, first expert, E, rows)"""
    if topk_ids.dim() != 2:
        raise ValueError(f"topk_ids: shape {tuple(topk_ids.shape)}, expected two dimensions")
    M, topk = topk_ids.shape
    begin = 0
    if expert_range is not None:
        begin, end = expert_range
        if not 0 <= begin < end <= E:
            raise ValueError(f"expert_range: {expert_range!r}, expected a part of [0, {E})")
        E = end - begin
    cap = rows(M, topk, E, block)
    if order is None:
        new = lambda *shape: _new(shape, torch.int32, topk_ids.device, stream)  # noqa: E731
        order = Order(new(E + 1), new(cap), new(M, topk))
    at = (_dense(order[0], torch.int32, (E + 1,), "order.offsets", dev),
          _dense(order[1], torch.int32, (cap,), "order.slots", dev),
          _dense(order[2], torch.int32, (M, topk), "order.position", dev))
    return order, at, M, topk, begin, E, cap


def sort(topk_ids, E, block=1, expert_range=None, order=None, stream=None) -> Order:
    """The order of the experts' rows for ``topk_ids`` int32 [M, topk] of ``E`` experts, each
    expert's rows filled up to a multiple of ``block``. With ``expert_range=(begin, end)``
    only those experts' (expert parallelism). Ids of no expert here get no row."""
    dev = _device(topk_ids, "topk_ids")
    order, at, M, topk, begin, E, _ = _order_for(topk_ids, E, block, expert_range, order, dev, stream)
    _check(lib().moe_w4a16_dispatch_sort(_dense(topk_ids, torch.int32, (M, topk), "topk_ids", dev), M, topk, begin, E,
                                         block, *at, _handle(stream, dev)))
    return order


def gather(x, order, out=None, stream=None):
    """``x`` [M, K] (bf16, fp32, e4m3 or bytes) in the order's rows: [rows, K]. Rows that fill
    up an expert's are 0, those behind the last expert's are left as they were (a new
    ``out`` is not cleared)."""
    if out is not None and stream is None and (fast := _fast(x)):
        calls, dev, handle = fast
        rc = calls.gather(dev, handle, x, *order, out)
        if rc is not None:
            _check(rc)
            return out
    M, K, stride = _rows(x, "x", _MOVED)
    dev = _device(x, "x")
    at, m, topk, E, cap, block = _parts(order, dev)
    if m != M:
        raise ValueError(f"order: of {m} tokens, x has {M}")
    if out is None:
        out = _new((cap, K), x.dtype, x.device, stream)
    _check(lib().moe_w4a16_dispatch_gather(x.data_ptr(), _MOVED[x.dtype], stride, *at,
                                           _dense(out, x.dtype, (cap, K), "out", dev), M, K, topk, E, block,
                                           _handle(stream, dev)))
    return out


def sort_gather(x, topk_ids, E, block=1, expert_range=None, out=None, order=None, stream=None):
    """``sort`` and ``gather`` in one call: ``(rows [rows, K], order)``."""
    if out is not None and order is not None and expert_range is None and stream is None and (fast := _fast(x)):
        calls, dev, handle = fast
        rc = calls.sort_gather(dev, handle, x, topk_ids, E, 0, block, *order, out)
        if rc is not None:
            _check(rc)
            return out, order
    M, K, stride = _rows(x, "x", _MOVED)
    dev = _device(x, "x")
    order, at, m, topk, begin, E, cap = _order_for(topk_ids, E, block, expert_range, order, dev, stream)
    if m != M:
        raise ValueError(f"topk_ids: of {m} tokens, x has {M}")
    if out is None:
        out = _new((cap, K), x.dtype, x.device, stream)
    _check(lib().moe_w4a16_dispatch_sort_gather(
        x.data_ptr(), _MOVED[x.dtype], stride, _dense(topk_ids, torch.int32, (M, topk), "topk_ids", dev), M, K, topk,
        begin, E, block, *at, _dense(out, x.dtype, (cap, K), "out", dev), _handle(stream, dev)))
    return out, order


def _combine(y, weights, order, add, out, out_dtype, stream):
    if out is not None and stream is None and (fast := _fast(y)):
        calls, dev, handle = fast
        rc = calls.combine(dev, handle, y, weights, order[1], order[2], add, out)
        if rc is not None:
            _check(rc)
            return out
    R, K, dev = _matrix(y, "y")
    _, slots, position = order
    if position.dim() != 2:
        raise ValueError(f"order.position: shape {tuple(position.shape)}, expected two dimensions")
    M, topk = position.shape
    at = _int32(position, "order.position", dev)
    if R != slots.shape[0]:
        raise ValueError(f"y: {R} rows, expected the order's {slots.shape[0]}")
    w = 0 if weights is None else _dense(weights, torch.float32, (M, topk), "weights", dev)
    if out is None:
        out = _new((M, K), out_dtype or y.dtype, y.device, stream)
    if out.dtype not in _FLOATS:
        raise ValueError(f"out: dtype {out.dtype}, expected one of {tuple(_FLOATS)}")
    plus = 0 if add is None else _dense(add, out.dtype, (M, K), "add", dev)
    _check(lib().moe_w4a16_combine(y.data_ptr(), _FLOATS[y.dtype], w, at, plus,
                                   _dense(out, out.dtype, (M, K), "out", dev), _FLOATS[out.dtype], M, K, topk, R,
                                   _handle(stream, dev)))
    return out


def combine(y, weights, order, add=None, out=None, out_dtype=None, stream=None):
    """The experts' rows ``y`` [rows, K] (bf16 or fp32) back to their tokens, with ``weights``
    fp32 [M, topk] and ``add`` [M, K] (of ``out``'s type, and may be ``out``): [M, K] in
    ``out_dtype`` (bf16 or fp32; by default that of ``y``)."""
    return _combine(y, weights, order, add, out, out_dtype, stream)


def gather_backward(drows, order, out=None, out_dtype=None, stream=None):
    """Gradient of ``gather``: the sum of each token's rows of ``drows`` [rows, K]: [M, K]."""
    return _combine(drows, None, order, None, out, out_dtype, stream)


def combine_backward(dout, y, weights, order, dy=None, dweights=None, stream=None):
    """Gradient of ``combine`` for ``dout`` [M, K]: ``(dy [rows, K] of y's type, dweights fp32
    [M, topk])``. Rows of ``dy`` that fill up an expert's are 0, those behind the last
    expert's are left as they were. ``add`` has the gradient ``dout`` itself."""
    if dy is not None and dweights is not None and stream is None and (fast := _fast(dout)):
        calls, dev, handle = fast
        rc = calls.combine_backward(dev, handle, dout, y, weights, *order, dy, dweights)
        if rc is not None:
            _check(rc)
            return dy, dweights
    M, K, dev = _matrix(dout, "dout")
    at, m, topk, E, cap, block = _parts(order, dev)
    if m != M:
        raise ValueError(f"order: of {m} tokens, dout has {M}")
    if y.dtype not in _FLOATS:
        raise ValueError(f"y: dtype {y.dtype}, expected one of {tuple(_FLOATS)}")
    src = _dense(y, y.dtype, (cap, K), "y", dev)
    w = _dense(weights, torch.float32, (M, topk), "weights", dev)
    if dy is None:
        dy = _new((cap, K), y.dtype, y.device, stream)
    if dweights is None:
        dweights = _new((M, topk), torch.float32, y.device, stream)
    _check(lib().moe_w4a16_combine_backward(
        dout.data_ptr(), _FLOATS[dout.dtype], src, _FLOATS[y.dtype], w, *at, _dense(dy, y.dtype, (cap, K), "dy", dev),
        _dense(dweights, torch.float32, (M, topk), "dweights", dev), M, K, topk, E, block, _handle(stream, dev)))
    return dy, dweights
