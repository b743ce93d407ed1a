"""A whole Mixture-of-Experts layer: the scored router, the W4A16 routed experts and the
8-bit shared expert, chained as a serving program does.

    ids, weights = route_scored(router_logits)          (selection: score + bias, groups)
    routed       = MoEW4A16.forward(hidden, ids, weights)
    out          = shared_expert(hidden) + routed       (added in fp32, rounded once)

With low-rank adapters of many requests beside the shared expert's gate/up product:

    [gate | up]  = quantize(hidden) . w1 + scale[l] b[l] (a[l] hidden)   (fp32; l: the row's adapter)
    out          = quantize(SiLU(gate) * up) . w2 + routed
"""
from __future__ import annotations

import torch

from . import MoEW4A16, fp8, lora, routing


class MoELayer:
    """Holds the routed experts (a packed ``MoEW4A16``), the router's settings and the
    shared expert's 8-bit weights ``(w1, w1_s, w2, w2_s)`` (see ``fp8.shared_expert``;
    ``None`` for a layer without one). ``adapters``: ``(a [L, r, K], b [L, 2 N, r])`` or ``(a, b,
    scale [L])`` of low-rank adapters beside its gate/up product (see ``lora.apply``; ``b``'s
    rows as ``w1``'s, gate then up)."""

    def __init__(self, experts: MoEW4A16, shared=None, scoring="sigmoid", bias=None, n_group=1, topk_group=1,
                 group_top=None, renormalize=True, scale=1.0, adapters=None):
        if experts.E != experts.E_total:
            raise ValueError("the layer needs all experts in one handle")
        if adapters is not None and shared is None:
            raise ValueError("adapters stand beside the shared expert, which the layer lacks")
        self.experts = experts
        self.adapters = adapters
        self.shared = shared
        self.router = dict(scoring=scoring, bias=bias, n_group=n_group, topk_group=topk_group, group_top=group_top,
                           renormalize=renormalize, scale=scale)

    def route(self, router_logits, stream=None):
        """``(ids, weights)`` of ``router_logits`` [M, E] (fp32 or bf16)."""
        return routing.route_scored(router_logits, self.experts.topk, stream=stream, **self.router)

    def _shared_with_adapters(self, hidden, adapter, out, stream):
        w1, w1_s, w2, w2_s = self.shared
        a, b, scale = (*self.adapters, None)[:3]
        gate_up = fp8.matmul(*fp8.quantize(hidden, stream=stream), w1, w1_s, out_dtype=torch.float32, stream=stream)
        lora.apply(hidden, a, b, adapter, add=gate_up, scale=scale, out=gate_up, stream=stream)
        fp8.matmul(*fp8.swiglu_quantize(gate_up, stream=stream), w2, w2_s, add=out, out=out, stream=stream)

    def forward(self, hidden, router_logits, out=None, stream=None, adapter=None):
        """``(out bf16 [M, K], ids, weights)`` of ``hidden`` bf16 [M, K]. ``adapter`` int32 [M]:
        the adapter of each row, -1 for none (needs a layer with ``adapters``)."""
        if router_logits.shape != (hidden.shape[0], self.experts.E_total):
            raise ValueError(f"router_logits: shape {tuple(router_logits.shape)}, expected "
                             f"{(hidden.shape[0], self.experts.E_total)}")
        if adapter is not None and self.adapters is None:
            raise ValueError("adapter: the layer has no adapters")
        ids, weights = self.route(router_logits, stream)
        out = self.experts.forward(hidden, ids, weights, out=out, stream=stream)
        if adapter is not None:
            self._shared_with_adapters(hidden, adapter, out, stream)
        elif self.shared is not None:
            fp8.shared_expert(hidden, *self.shared, add=out, out=out, stream=stream)
        return out, ids, weights
