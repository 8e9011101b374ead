"""Runs a small latent sparse block with sigmoid routing, a balance bias and expert groups, then tunes its router over the frozen
4-bit experts towards the outputs of another router.

    python examples/latent_block.py [--steps 60] [--tokens 512]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_expert_ffn_moe_gb300 import binding as B  # noqa: E402
from bit_expert_ffn_moe_gb300 import inputs as IN  # noqa: E402
from bit_expert_ffn_moe_gb300 import ops  # noqa: E402
from bit_expert_ffn_moe_gb300.block import LatentBlock  # noqa: E402
from bit_expert_ffn_moe_gb300.layer import DeviceLayer  # noqa: E402


def build(tokens: int, D: int = 1024, seed: int = 0, wfmt: str = "nvfp4") -> LatentBlock:
    cfg = IN.small_config("latent_block", T=tokens, d=512, E=16, k=4, I=256, index=190)
    g = torch.Generator(device="cuda").manual_seed(seed)
    W_in = (torch.randn(cfg.d, D, generator=g, device="cuda") / D ** 0.5).bfloat16()
    W_out = (torch.randn(D, cfg.d, generator=g, device="cuda") / cfg.d ** 0.5).bfloat16()
    rule = ops.route_rule("sigmoid", groups=4, top_groups=2, group_score="top2", renormalize=True, scale=2.0)
    return LatentBlock(DeviceLayer(cfg, wfmt=wfmt), rule, W_in, W_out, tokens, torch.zeros(cfg.E, device="cuda"), gradients=True)


def tune(block: LatentBlock, x: torch.Tensor, target: torch.Tensor, steps: int, rate: float, say=None) -> list:
    """Gradient descent of mean |y - target|^2 over the router alone; the losses."""
    losses = []
    for i in range(steps):
        y, past = block(x)
        diff = y.float() - target.float()
        losses.append(float((diff ** 2).mean()))
        grad = block.router_gradient((diff / diff.abs().max()).bfloat16(), past)
        block.W_r -= rate * grad / grad.norm().clamp_min(1e-20)
        if say and (i % 10 == 0 or i == steps - 1):
            say("step %3d  loss %.5f" % (i, losses[-1]))
    return losses


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    block = build(a.tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, block.narrow.K, generator=g, device="cuda").bfloat16()
    target, _ = block(x)
    load = block.counts.float()
    print("picks per expert: mean %.0f, largest %.0f" % (load.mean(), load.max()))
    for _ in range(40):
        block(x)
        block.balance_step(0.002)
    load = block.counts.float()
    print("after 40 balance steps: largest %.0f" % load.max())
    block.balance.zero_()
    block.W_r += 0.5 * torch.randn(block.W_r.shape, generator=g, device="cuda") / block.layer.cfg.d ** 0.5
    losses = tune(block, x, target, a.steps, 0.3, print)
    print("loss %.5f -> %.5f" % (losses[0], losses[-1]))
    if B.moe_get_device_status(block.ws) != B.MOE_OK:
        raise SystemExit("device status")


if __name__ == "__main__":
    main()
