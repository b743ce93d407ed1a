"""One Mixture-of-Experts layer on random weights: route, routed experts, shared expert.

    python examples/moe_layer.py [--tokens 64] [--experts 64] [--hidden 1024] [--inter 512]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

from int4_weight_only_moe_gb300 import MoEW4A16, fp8, inputs
from int4_weight_only_moe_gb300.layer import MoELayer


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inter", type=int, default=512)
    ap.add_argument("--topk", type=int, default=8)
    a = ap.parse_args()
    E, K, N = a.experts, a.hidden, a.inter

    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()
    w1_q, w1_s, w2_q, w2_s = inputs.all_expert_weights(E, K, N)
    experts = MoEW4A16(E, K, N, a.topk)
    experts.pack(dev(w1_q), dev(w1_s.view(np.int16)), dev(w2_q), dev(w2_s.view(np.int16)))

    g = torch.Generator(device="cuda").manual_seed(0)
    normal = lambda *shape, by: (torch.randn(*shape, generator=g, device="cuda") * by).bfloat16()
    shared = fp8.quantize_weight(normal(2 * N, K, by=K ** -0.5)) + fp8.quantize_weight(normal(K, N, by=N ** -0.5))
    gate = normal(E, K, by=K ** -0.5)
    groups = 8 if E % 8 == 0 and a.topk <= E // 2 else 1
    layer = MoELayer(experts, shared, scoring="sigmoid", bias=torch.zeros(E, device="cuda"), n_group=groups,
                     topk_group=max(1, groups // 2), scale=2.5)

    hidden = normal(a.tokens, K, by=1.0)
    out, ids, weights = layer.forward(hidden, hidden @ gate.t())
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, {E} experts, top-{a.topk}: out {tuple(out.shape)} {out.dtype}, "
          f"rms {out.float().square().mean().sqrt():.3f}, status {experts.status()} / {fp8.status()}")
    print("first token's experts", ids[0].tolist(), "weights", [round(w, 3) for w in weights[0].tolist()])
    experts.close()


if __name__ == "__main__":
    main()
