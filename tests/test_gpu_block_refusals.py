"""Calls of a latent block that was built without what they need."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gradients_and_balance_have_to_be_asked_for():
    import latent_block as example
    from bit_expert_ffn_moe_gb300.block import LatentBlock
    whole = example.build(4)
    W_in, W_out = (torch.randn(s, device="cuda").bfloat16() for s in ((512, 1024), (1024, 512)))
    block = LatentBlock(whole.layer, whole.rule, W_in, W_out, 4)
    y, past = block(torch.randn(4, 1024, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="without gradients"):
        block.router_gradient(y, past)
    with pytest.raises(ValueError, match="without a balance bias"):
        block.balance_step(0.1)
    with pytest.raises(ValueError, match="at most 4 tokens"):
        block(torch.randn(5, 1024, device="cuda").bfloat16())


def test_no_tokens():
    import latent_block as example
    block = example.build(4)
    y, past = block(torch.empty(0, 1024, device="cuda").bfloat16())
    assert y.shape == (0, 1024) and int(block.counts.sum()) == 0
    assert (block.router_gradient(y, past) == 0).all()
