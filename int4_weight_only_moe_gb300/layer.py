"""A whole Mixture-of-Experts layer: the scored router, the W4A16 routed experts and the
8-bit shared expert, chained as a serving program does.

    ids, weights = route_scored(router_logits)          (selection: score + bias, groups)
    routed       = MoEW4A16.forward(hidden, ids, weights)
    out          = shared_expert(hidden) + routed       (added in fp32, rounded once)
"""
from __future__ import annotations

from . import MoEW4A16, fp8, routing


class MoELayer:
    """Holds the routed experts (a packed ``MoEW4A16``), the router's settings and the
    shared expert's 8-bit weights ``(w1, w1_s, w2, w2_s)`` (see ``fp8.shared_expert``;
    ``None`` for a layer without one)."""

    def __init__(self, experts: MoEW4A16, shared=None, scoring="sigmoid", bias=None, n_group=1, topk_group=1,
                 group_top=None, renormalize=True, scale=1.0):
        if experts.E != experts.E_total:
            raise ValueError("the layer needs all experts in one handle")
        self.experts = experts
        self.shared = shared
        self.router = dict(scoring=scoring, bias=bias, n_group=n_group, topk_group=topk_group, group_top=group_top,
                           renormalize=renormalize, scale=scale)

    def route(self, router_logits, stream=None):
        """``(ids, weights)`` of ``router_logits`` [M, E] (fp32 or bf16)."""
        return routing.route_scored(router_logits, self.experts.topk, stream=stream, **self.router)

    def forward(self, hidden, router_logits, out=None, stream=None):
        """``(out bf16 [M, K], ids, weights)`` of ``hidden`` bf16 [M, K]."""
        if router_logits.shape != (hidden.shape[0], self.experts.E_total):
            raise ValueError(f"router_logits: shape {tuple(router_logits.shape)}, expected "
                             f"{(hidden.shape[0], self.experts.E_total)}")
        ids, weights = self.route(router_logits, stream)
        out = self.experts.forward(hidden, ids, weights, out=out, stream=stream)
        if self.shared is not None:
            fp8.shared_expert(hidden, *self.shared, add=out, out=out, stream=stream)
        return out, ids, weights
