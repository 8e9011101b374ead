"""Runs a sparse layer with 8-bit experts behind a sigmoid routing rule, and tunes its router over the frozen experts towards the outputs
of another router.

    python examples/int8_experts.py [--steps 60] [--tokens 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_expert_ffn_moe_gb300 import binding as B  # noqa: E402
from bit_expert_ffn_moe_gb300 import ops  # noqa: E402
from bit_expert_ffn_moe_gb300.block import Int8Experts  # noqa: E402


class Layer:
    def __init__(self, tokens: int, d: int = 512, E: int = 16, k: int = 4, I: int = 256, seed: int = 0):  # noqa: E741
        g = torch.Generator(device="cuda").manual_seed(seed)

        def matrices(n, m):
            return torch.randn(E, n, m, generator=g, device="cuda") / m ** 0.5
        self.experts = Int8Experts(ops.int8_weights(matrices(I, d), up=matrices(I, d)), ops.int8_weights(matrices(d, I)), tokens, k)
        self.W_r = torch.randn(E, d, generator=g, device="cuda") / d ** 0.5
        self.rule, self.k, self.d = ops.route_rule("sigmoid", renormalize=True, scale=2.0), k, d

    def route(self, x: torch.Tensor):
        logits = ops.route_logits(x, self.W_r)
        return (logits, *ops.route_scores(logits, self.k, self.rule))

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        _, ids, w = self.route(x)
        return self.experts(x, ids, w)

    def forward_and_gradient(self, x: torch.Tensor, gradient_of):
        """y, and the gradient of W_r for dy = gradient_of(y)."""
        logits, ids, w = self.route(x)
        rows, order = self.experts.outputs(x, ids)
        y = ops.experts_to_tokens(rows, order, w)
        _, dw = ops.experts_to_tokens_backward(gradient_of(y), order, rows, w, need_drows=False)
        dlogits = ops.route_scores_backward(logits, ids, dw, self.rule)
        return y, dlogits.t() @ x.float()


def tune(layer: Layer, x: torch.Tensor, target: torch.Tensor, steps: int, rate: float, say=None) -> list:
    """Gradient descent of mean |y - target|^2 over the router alone; the losses."""
    losses = []
    for i in range(steps):
        y, grad = layer.forward_and_gradient(x, lambda y: ((y.float() - target.float()) / y.numel()).to(y.dtype))
        losses.append(float(((y.float() - target.float()) ** 2).mean()))
        layer.W_r -= rate * grad / grad.norm().clamp_min(1e-20)
        if say and (i % 10 == 0 or i == steps - 1):
            say("step %3d  loss %.5f" % (i, losses[-1]))
    return losses


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    layer = Layer(a.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, layer.d, generator=g, device="cuda").bfloat16()
    target = layer(x)
    layer.W_r += 0.5 * torch.randn(layer.W_r.shape, generator=g, device="cuda") / layer.d ** 0.5
    losses = tune(layer, x, target, a.steps, 0.3, print)
    print("loss %.5f -> %.5f" % (losses[0], losses[-1]))
    if B.moe_get_device_status(layer.experts.workspace) != B.MOE_OK:
        raise SystemExit("device status")


if __name__ == "__main__":
    main()
