"""Low-rank adapters of many requests beside a projection (definition: ``moe_w4a16_lora``
in ``include/moe_w4a16.h``)."""
from __future__ import annotations

import functools

import torch

from . import BF16, F32, _check, _new, lib, moe_w4a16_lora_workspace_size
from .routing import _dense, _device, _fast, _handle, _on, _rows

_FLOATS = {torch.float32: F32, torch.bfloat16: BF16}
_POOL_BYTES = 16 << 20
_workspace_size = functools.lru_cache(maxsize=256)(moe_w4a16_lora_workspace_size)


def apply(x, a, b, index, add=None, scale=None, out=None, out_dtype=torch.bfloat16, workspace=None, stream=None):
    """``add[m] + scale[l] b[l] (a[l] x[m])`` with ``l = index[m]``, ``add[m]`` where that is no
    adapter (-1): [M, N] in ``out_dtype`` (bf16 or fp32; that of ``out`` where it is given).

    ``x`` bf16 [M, K]; ``a`` bf16 [L, r, K]; ``b`` bf16 [L, N, r]; ``index`` int32 [M]; ``scale``
    fp32 [L] (None: 1); ``add`` bf16 or fp32 [M, N], the projection's output (``fp8.matmul``;
    None: 0), which ``out`` may be. ``workspace``: uint8, of
    ``moe_w4a16_lora_workspace_size(M, K, N, r, L)`` bytes; where it is not given, up to 16
    MiB come from the library's stream-ordered pool, more from torch.
    """
    if out is not None and workspace is None and stream is None and (fast := _fast(x)):
        calls, dev, handle = fast
        rc = calls.lora(dev, handle, x, a, b, index, add, scale, out, _POOL_BYTES)
        if rc is not None:
            _check(rc)
            return out
    M, K, ldx = _rows(x, "x", (torch.bfloat16,))
    dev = _device(x, "x")
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a and b: expected [L, r, K] and [L, N, r]")
    L, r, _ = a.shape
    N = b.shape[1]
    pa = _dense(a, torch.bfloat16, (L, r, K), "a", dev)
    pb = _dense(b, torch.bfloat16, (L, N, r), "b", dev)
    i = _dense(index, torch.int32, (M,), "index", dev)
    s = 0 if scale is None else _dense(scale, torch.float32, (L,), "scale", dev)
    if out is None:
        out = _new((M, N), out_dtype, x.device, stream)
    if out.dtype not in _FLOATS:
        raise ValueError(f"out: dtype {out.dtype}, expected one of {tuple(_FLOATS)}")
    plus, kind = 0, F32
    if add is not None:
        if add.dtype not in _FLOATS:
            raise ValueError(f"add: dtype {add.dtype}, expected one of {tuple(_FLOATS)}")
        plus, kind = _dense(add, add.dtype, (M, N), "add", dev), _FLOATS[add.dtype]
    if workspace is None and (need := _workspace_size(M, K, N, r, L)) > _POOL_BYTES:
        workspace = _new((need,), torch.uint8, x.device, stream)
    ws = size = 0
    if workspace is not None:
        _on(workspace, dev, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        ws, size = workspace.data_ptr(), workspace.nbytes
    _check(lib().moe_w4a16_lora(x.data_ptr(), ldx, pa, pb, s, i, plus, kind,
                                _dense(out, out.dtype, (M, N), "out", dev), _FLOATS[out.dtype], M, K, N, r, L, ws, size,
                                _handle(stream, dev)))
    return out
