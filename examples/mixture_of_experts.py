"""One feed-forward half of a mixture-of-experts layer, with this library's operators.

A router's logits choose each token's experts (moe_route); the chosen experts'
gated MXFP4 products are weighted and added to the layer's input (mxfp4_moe);
a shared expert that every token passes is two linears, the first with its
gate (mxfp4_linear_act), the second adding its result to the same rows.

    python examples/mixture_of_experts.py [--tokens 200] [--hidden 1024] [--shards 2]

prints the largest difference between the layer in one piece and the sum of
its shards, each of which holds a run of the experts and leaves out the
others' (ids outside its own add nothing).
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp4_block_scaled_quant_amd as mx  # noqa: E402


class MixtureOfExperts:
    """E gated experts of ``inner`` values, ``top_k`` a token, and a shared one."""

    def __init__(self, router: torch.Tensor, bias: torch.Tensor, up: torch.Tensor, down: torch.Tensor,
                 shared_up: torch.Tensor, shared_down: torch.Tensor, top_k: int, groups: int, top_groups: int):
        # router [E, hidden], bias fp32 [E]; up [E, 2 inner, hidden] (gate first), down [E, hidden, inner];
        # shared_up [2 inner, hidden], shared_down [hidden, inner]
        self.router, self.bias = router, bias
        self.up, self.down = mx.quantize_weight(up), mx.quantize_weight(down)
        self.shared_up, self.shared_down = mx.quantize_weight(shared_up), mx.quantize_weight(shared_down)
        self.top_k, self.groups, self.top_groups = top_k, groups, top_groups

    def choose(self, x: torch.Tensor):
        logits = (x @ self.router.T).float()
        return mx.moe_route(logits, self.top_k, self.bias, scoring="sigmoid", groups=self.groups,
                            top_groups=self.top_groups, scale=2.5)

    def shared(self, x: torch.Tensor, onto: torch.Tensor) -> torch.Tensor:
        """onto + the shared expert of x, written where onto stands."""
        h = mx.mxfp4_linear_act(x, self.shared_up.w_pre, self.shared_up.ws_pre, self.shared_up.N, activation="silu",
                                gated=True)
        return mx.mxfp4_linear_act(h, self.shared_down.w_pre, self.shared_down.ws_pre, self.shared_down.N,
                                   residual=onto, out=onto)

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        weights, ids = self.choose(x)
        return self.shared(x, mx.mxfp4_moe(x, ids, weights, self.up, self.down, residual=x))

    def shard(self, x: torch.Tensor, first: int, experts: int) -> torch.Tensor:
        """The routed part of experts [first, first + experts), as the process that holds them computes it."""
        weights, ids = self.choose(x)
        cut = lambda w: mx.MXFP4Weight(  # noqa: E731
            w.w_pre.reshape(w.batch, -1)[first:first + experts].reshape(-1),
            w.ws_pre.reshape(w.batch, -1)[first:first + experts].reshape(-1), w.N, w.K, experts)
        return mx.mxfp4_moe(x, ids - first, weights, cut(self.up), cut(self.down))


def build(hidden: int, inner: int, experts: int, top_k: int, groups: int, top_groups: int, device: str = "cuda"):
    g = torch.Generator(device=device).manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    rows = lambda *s: (randn(*s) / s[-1] ** 0.5).to(torch.bfloat16)  # noqa: E731
    return MixtureOfExperts(rows(experts, hidden), randn(experts) * 0.05, rows(experts, 2 * inner, hidden),
                            rows(experts, hidden, inner), rows(2 * inner, hidden), rows(hidden, inner), top_k, groups,
                            top_groups)


def demo(tokens: int = 200, hidden: int = 1024, inner: int = 512, experts: int = 32, top_k: int = 4, groups: int = 4,
         top_groups: int = 2, shards: int = 2, device: str = "cuda"):
    """Runs the layer; returns the largest difference of the shards' sum and the largest value on the way."""
    layer = build(hidden, inner, experts, top_k, groups, top_groups, device)
    x = torch.randn(tokens, hidden, generator=torch.Generator(device=device).manual_seed(2),
                    device=device).to(torch.bfloat16)
    whole = layer(x)
    own = experts // shards
    parts = [layer.shard(x, i * own, own).float() for i in range(shards)]
    mixed = x.float() + sum(parts)
    top = max(t.abs().max().item() for t in (mixed, whole.float(), *parts))
    summed = layer.shared(x, mixed.to(torch.bfloat16))
    torch.cuda.synchronize()
    return (whole.float() - summed.float()).abs().max().item(), top


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--shards", type=int, default=2)
    args = ap.parse_args()
    off, top = demo(args.tokens, args.hidden, shards=args.shards)
    print(f"values up to {top:.3g}; the shards' sum off by {off:.3g} at most")
