"""The routing rules, NVFP4 projections and their gradients together, as a latent sparse block runs them."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 37, 300])
def test_forward_is_its_parts(tokens):
    """The plain softmax rule chooses and weighs like the layer call's router, so block = projection, layer call, projection; the
    expert outputs are the same kernels', the weights differ in their last bits, one bf16 rounding lies between."""
    from bit_expert_ffn_moe_gb300 import binding as B
    from bit_expert_ffn_moe_gb300 import ops
    from bit_expert_ffn_moe_gb300.layer import layer_forward, make_workspace
    import latent_block as example
    block = example.build(300)
    block.rule = ops.route_rule("softmax")
    block.balance = None
    x = torch.randn(tokens, 1024, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    y, past = block(x)
    cfg = block.layer.cfg
    block.layer.b.zero_()
    ws = make_workspace(tokens, cfg.d, cfg.E, cfg.k, cfg.I, B.MOE_ACT_MXFP4)
    s, ids, w = layer_forward(block.layer, past["z"], B.MOE_ACT_MXFP4, ws=ws, want_routing=True)
    assert torch.equal(ids, past["ids"])
    assert (w - past["w"]).abs().max() <= 2.0 ** -20
    want = block.widen(s)
    assert torch.linalg.norm((y - want).float()) <= 2.0 ** -8 * torch.linalg.norm(want.float())
    for ws_ in (block.ws, block.narrow.workspace, block.widen.workspace):
        assert B.moe_get_device_status(ws_) == B.MOE_OK


def test_router_gradient_against_autograd():
    """dW_r against 64-bit autograd of the same frozen pass: choice and expert outputs held, dy as its quantised values.  The chain rounds
    ds to bf16 (2^-8 relative, uncorrelated between the d = 512 terms of each dw) and dw, dlogits in fp32."""
    from bit_expert_ffn_moe_gb300 import ops
    import latent_block as example
    block = example.build(200)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(200, 1024, generator=g, device="cuda").bfloat16()
    y, past = block(x)
    dy = torch.randn(y.shape, generator=g, device="cuda").bfloat16()
    got = block.router_gradient(dy, past)
    q = ops.nvfp4_operand(*dy.shape)
    ops.nvfp4_quantize(dy, q)
    W_r = block.W_r.double().requires_grad_(True)
    z, ids, T, k = past["z"].double(), past["ids"].long(), 200, block.layer.cfg.k
    u = torch.sigmoid(z @ W_r.T).gather(1, ids)
    w = block.rule.scale * u / u.sum(1, keepdim=True)
    rows = past["y_perm"].double()[past["inv"].long()].view(T, k, -1)
    s = (w[:, :, None] * rows).sum(1)
    ((s @ block.widen.transposed.values().double()) * q.values().double()).sum().backward()
    assert torch.linalg.norm(got.double() - W_r.grad) <= 2.0 ** -8 * torch.linalg.norm(W_r.grad)


def test_tuning_lowers_the_loss():
    import latent_block as example
    block = example.build(256)
    g = torch.Generator(device="cuda").manual_seed(7)
    x = torch.randn(256, 1024, generator=g, device="cuda").bfloat16()
    target, _ = block(x)
    block.W_r += 0.5 * torch.randn(block.W_r.shape, generator=g, device="cuda") / block.layer.cfg.d ** 0.5
    losses = example.tune(block, x, target, 25, 0.3)
    assert losses[-1] < 0.7 * losses[0]
