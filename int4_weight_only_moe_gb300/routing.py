"""Router with scores, a balance bias and expert groups, in front of the routed experts.

``route_scored`` turns the gate's logits into the ``topk_ids`` and ``topk_weights`` that
``MoEW4A16.forward`` takes (definition: ``moe_w4a16_route_scored`` in
``include/moe_w4a16.h``). ``MoEW4A16.route`` is the plain form, a softmax over the
selected logits.
"""
from __future__ import annotations

import torch

from . import BF16, F32, SCORE_SIGMOID, SCORE_SOFTMAX, _check, _need, _new, lib

_SCORES = {"sigmoid": SCORE_SIGMOID, "softmax": SCORE_SOFTMAX}
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _rows(t, name, types):
    """(rows, columns, row stride) of a 2-D CUDA tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected two dimensions")
    if t.dtype not in types:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(types)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    (rows, cols), (stride, inner) = t.shape, t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    if stride < cols:
        if rows > 1:
            raise ValueError(f"{name}: rows overlap (stride {stride}, {cols} values)")
        stride = cols
    return rows, cols, stride


def _device(t, name):
    """Index of the device of ``t``, which has to be the current one: that is where the
    library launches."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {t.device}, the current device is cuda:{torch._C._cuda_getDevice()}")
    return dev


def _on(t, dev, name):
    """Refuses a tensor that is not on device ``dev``."""
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")


def _dense(t, dtype, shape, name, dev):
    """``t`` itself, when it is a contiguous tensor of this type and shape on device
    ``dev``; its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        _need(t, (str(dtype).removeprefix("torch."),), shape, name)
        _on(t, dev, name)
    return t.data_ptr()


def _handle(stream, dev):
    """Raw handle of ``stream``, or of the current stream of device ``dev``."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return int(getattr(stream, "cuda_stream", stream))


def route_scored(logits, topk, scoring="sigmoid", bias=None, n_group=1, topk_group=1, group_top=None,
                 renormalize=True, scale=1.0, ids=None, weights=None, stream=None):
    """Scores, biased and group-limited top-k and weights of ``logits`` [M, E] (fp32 or
    bf16): ``(ids int32 [M, topk], weights fp32 [M, topk])``.

    ``bias`` fp32 [E] takes part in the selection only. ``group_top`` (1 or 2) is how many
    of a group's largest values count for it; by default 2 with a bias, 1 without.
    """
    M, E, stride = _rows(logits, "logits", _TYPES)
    dev = _device(logits, "logits")
    score = _SCORES.get(scoring)
    if score is None:
        raise ValueError(f"scoring: {scoring!r}, expected one of {tuple(_SCORES)}")
    b = 0 if bias is None else _dense(bias, torch.float32, (E,), "bias", dev)
    if group_top is None:
        group_top = 2 if bias is not None else 1
    if ids is None:
        ids = _new((M, topk), torch.int32, logits.device, stream)
    if weights is None:
        weights = _new((M, topk), torch.float32, logits.device, stream)
    _check(lib().moe_w4a16_route_scored(
        logits.data_ptr(), _TYPES[logits.dtype], stride, M, E, topk, score, b, n_group, topk_group, group_top,
        renormalize, scale, _dense(ids, torch.int32, (M, topk), "ids", dev),
        _dense(weights, torch.float32, (M, topk), "weights", dev), _handle(stream, dev)))
    return ids, weights
