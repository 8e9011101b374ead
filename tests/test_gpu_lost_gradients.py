"""Products of operands that were made of a tensor which requires a gradient: backward() through them is an error, as it is for the calls that
take the tensor itself, and not a gradient that lacks their part."""
import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops
from bit_expert_ffn_moe_gb300.block import Int8Experts

pytestmark = pytest.mark.gpu


def int8_forms():
    """Name, input, and the differentiable result of it."""
    g = torch.Generator(device="cuda").manual_seed(0)
    ids = R.some_ids(6, 3, 8, 1).cuda()
    order = ops.expert_order(ids, 8)
    x, rows = torch.randn(6, 64, generator=g, device="cuda"), torch.randn(18, 64, generator=g, device="cuda")
    W, We = ops.int8_weights(torch.randn(40, 64, generator=g, device="cuda")), ops.int8_weights(torch.randn(8, 40, 64, generator=g, device="cuda"))
    ws = ops.int8_workspace(18, 40, 64)
    up = ops.int8_weights(torch.randn(8, 32, 64, generator=g, device="cuda"), up=torch.randn(8, 32, 64, generator=g, device="cuda"))
    layer = Int8Experts(up, ops.int8_weights(torch.randn(8, 64, 32, generator=g, device="cuda")), 6, 3, torch.float32)
    w = torch.rand(6, 3, generator=g, device="cuda")
    yield "matmul", x, lambda t: ops.int8_matmul(ops.int8_quantize(t), W, torch.float32, ws)
    yield "gated", x, lambda t: ops.int8_matmul(ops.int8_quantize(t), W, torch.float32, ws, gated=True)
    yield "spread by expert", x, lambda t: ops.int8_matmul(ops.int8_quantize(t, order), We, torch.float32, ws)
    yield "in expert order", rows, lambda t: ops.int8_matmul(ops.int8_quantize(t, order, ordered=True), We, torch.float32, ws)
    yield "Int8Experts.outputs", x, lambda t: layer.outputs(t, ids)[0]
    yield "their sum", x, lambda t: ops.experts_to_tokens(layer.outputs(t, ids)[0], order, w)


def nvfp4_operand_of(t, columns=False):
    op, ws = ops.nvfp4_operand(*(t.t() if columns else t).shape), ops.nvfp4_workspace(*t.shape, 1)
    ops.nvfp4_quantize(t, None if columns else op, op if columns else None, ws)
    return op


def nvfp4_forms():
    g = torch.Generator(device="cuda").manual_seed(1)
    x, y = torch.randn(6, 64, generator=g, device="cuda"), torch.randn(40, 64, generator=g, device="cuda")
    ws = ops.nvfp4_workspace(64, 64, 64)
    yield "first", x, lambda t: ops.nvfp4_matmul(nvfp4_operand_of(t), nvfp4_operand_of(y), torch.float32, ws)
    yield "second", y, lambda t: ops.nvfp4_matmul(nvfp4_operand_of(x), nvfp4_operand_of(t), torch.float32, ws)
    yield "of columns", x, lambda t: ops.nvfp4_matmul(nvfp4_operand_of(t, True), nvfp4_operand_of(x, True), torch.float32, ws)


def check(forms):
    for name, x, f in forms:
        plain = f(x)
        assert not plain.requires_grad, name
        leaf = x.clone().requires_grad_(True)
        with torch.no_grad():
            assert not f(leaf).requires_grad, name
        y = f(leaf)
        assert torch.equal(y, plain), name
        with pytest.raises(RuntimeError, match="no autograd formula"):
            (leaf.sum() + y.sum()).backward()
        assert leaf.grad is None, name


def test_int8_operands():
    check(int8_forms())


def test_int8_operands_made_without_a_graph_are_constants():
    x = torch.randn(6, 64, device="cuda", requires_grad=True)
    W, ws = ops.int8_weights(torch.randn(40, 64, device="cuda")), ops.int8_workspace(6, 40, 64)
    with torch.no_grad():
        rows = ops.int8_quantize(x)
    assert not ops.int8_matmul(rows, W, torch.float32, ws).requires_grad
    out = torch.empty(6, 40, device="cuda")
    y = ops.int8_matmul(ops.int8_quantize(x), W, torch.float32, ws, out=out)
    assert y.data_ptr() == out.data_ptr() and not y.requires_grad and not out.requires_grad


def test_nvfp4_operands():
    check(nvfp4_forms())


def test_an_nvfp4_operand_is_what_it_was_last_made_of():
    x, ws = torch.randn(6, 64, device="cuda", requires_grad=True), ops.nvfp4_workspace(64, 64, 64)
    op, other = nvfp4_operand_of(x), nvfp4_operand_of(torch.randn(8, 64, device="cuda"))
    assert ops.nvfp4_matmul(op, other, torch.float32, ws).requires_grad
    ops.nvfp4_quantize(x.detach(), op)
    assert not ops.nvfp4_matmul(op, other, torch.float32, ws).requires_grad
    out = torch.empty(6, 8, device="cuda")
    assert not ops.nvfp4_matmul(nvfp4_operand_of(x), other, torch.float32, ws, out).requires_grad and not out.requires_grad
