"""Router with scores, a balance bias and expert groups, in front of the routed experts.

``route_scored`` turns the gate's logits into the ``topk_ids`` and ``topk_weights`` that
``MoEW4A16.forward`` takes (definition: ``moe_w4a16_route_scored`` in
``include/moe_w4a16.h``). ``MoEW4A16.route`` is the plain form, a softmax over the
selected logits.
"""
from __future__ import annotations

import torch

from . import BF16, F32, SCORE_SIGMOID, SCORE_SOFTMAX, _need, moe_w4a16_route_scored

_SCORES = {"sigmoid": SCORE_SIGMOID, "softmax": SCORE_SOFTMAX}
_TYPES = {torch.float32: F32, torch.bfloat16: BF16}


def _rows(t, name, types):
    """Row stride of a 2-D CUDA tensor whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected two dimensions")
    if t.dtype not in types:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {tuple(types)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    stride = t.stride(0)
    if rows <= 1:
        return max(stride, cols)
    if stride < cols:
        raise ValueError(f"{name}: rows overlap (stride {stride}, {cols} values)")
    return stride


def _lend(stream, *tensors):
    """Tell the allocator that ``stream``, when not the current one, uses new tensors."""
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
        for t in tensors:
            t.record_stream(s)


def route_scored(logits, topk, scoring="sigmoid", bias=None, n_group=1, topk_group=1, group_top=None,
                 renormalize=True, scale=1.0, ids=None, weights=None, stream=None):
    """Scores, biased and group-limited top-k and weights of ``logits`` [M, E] (fp32 or
    bf16): ``(ids int32 [M, topk], weights fp32 [M, topk])``.

    ``bias`` fp32 [E] takes part in the selection only. ``group_top`` (1 or 2) is how many
    of a group's largest values count for it; by default 2 with a bias, 1 without.
    """
    stride = _rows(logits, "logits", _TYPES)
    M, E = logits.shape
    if scoring not in _SCORES:
        raise ValueError(f"scoring: {scoring!r}, expected one of {tuple(_SCORES)}")
    if bias is not None:
        _need(bias, ("float32",), (E,), "bias")
    if group_top is None:
        group_top = 2 if bias is not None else 1
    if ids is None:
        ids = torch.empty((M, topk), dtype=torch.int32, device=logits.device)
        _lend(stream, ids)
    else:
        _need(ids, ("int32",), (M, topk), "ids")
    if weights is None:
        weights = torch.empty((M, topk), dtype=torch.float32, device=logits.device)
        _lend(stream, weights)
    else:
        _need(weights, ("float32",), (M, topk), "weights")
    moe_w4a16_route_scored(logits, _TYPES[logits.dtype], stride, M, E, topk, _SCORES[scoring], bias, n_group,
                           topk_group, group_top, bool(renormalize), scale, ids, weights, stream)
    return ids, weights
