"""The calls compute no autograd graph: where an input requires a gradient, backward() through their results is an error and not a
gradient that lacks their part."""
import os
import sys

import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def forms():
    """Name, input, and the differentiable result of it."""
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(4, 256, generator=g, device="cuda").bfloat16()
    W = ops.nvfp4_operand(256, 256)
    ops.nvfp4_quantize(torch.randn(256, 256, generator=g, device="cuda"), W)
    ws = ops.nvfp4_workspace(4, 256, 256)
    W_r = torch.randn(16, 256, generator=g, device="cuda")
    yield "scores", torch.randn(4, 64, generator=g, device="cuda"), lambda t: ops.route_scores(t, 4, ops.route_rule())[1]
    yield "linear", x, lambda t: ops.nvfp4_linear(t, W, ws)
    yield "logits of x", x, lambda t: ops.route_logits(t, W_r)
    yield "logits of W_r", W_r, lambda t: ops.route_logits(x, t)
    import latent_block as example
    block = example.build(4)
    yield "block", torch.randn(4, 1024, generator=g, device="cuda").bfloat16(), lambda t: block(t)[0]


def test_backward_is_an_error_where_a_gradient_would_be_lost():
    for name, x, f in forms():
        plain = f(x)
        assert not plain.requires_grad, name
        leaf = x.clone().requires_grad_(True)
        with torch.no_grad():
            assert not f(leaf).requires_grad, name
        y = f(leaf)
        assert torch.equal(y, plain), name
        with pytest.raises(RuntimeError, match="no autograd formula"):
            (leaf.float().sum() + y.float().sum()).backward()  # (without y's part, ones)
        assert leaf.grad is None, name


def test_results_of_the_gradient_calls_are_constants():
    logits = torch.randn(4, 64, device="cuda", requires_grad=True)
    rule = ops.route_rule()
    ids, w = ops.route_scores(logits, 4, rule)
    dlogits = ops.route_scores_backward(logits, ids, w, rule)
    assert not dlogits.requires_grad
    logits.backward(dlogits)
    assert torch.equal(logits.grad, dlogits)


def test_results_in_given_tensors_stay_what_they_are():
    x = torch.randn(4, 256, device="cuda", requires_grad=True)
    W = ops.nvfp4_operand(32, 256)
    ops.nvfp4_quantize(torch.randn(32, 256, device="cuda"), W)
    out = torch.empty(4, 32, device="cuda")
    y = ops.nvfp4_linear(x, W, ops.nvfp4_workspace(4, 32, 256), out)
    assert y.data_ptr() == out.data_ptr() and not y.requires_grad and not out.requires_grad


def test_the_blocks_router_gradient_is_a_constant():
    import latent_block as example
    block = example.build(8)
    x = torch.randn(8, 1024, device="cuda").bfloat16().requires_grad_(True)
    y, past = block(x)
    assert y.requires_grad and not any(t.requires_grad for t in past.values())
    grad = block.router_gradient(y.float().bfloat16(), past)
    assert not grad.requires_grad
    block.W_r -= grad
    assert not block.W_r.requires_grad
