"""Refusals of the routing rules, the weighted sum's gradients and the NVFP4 products beyond those of null pointers and shapes."""
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

INVALID = B.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("off", [1, 2, 3])
def test_arrays_of_words_start_on_four_bytes(off):
    """Floats and ints at odd places would fault on the GPU: refused before a launch, one argument at a time."""
    lib, bad = B.load(), 256 + off

    def scores(bias=256, ids=256, w=256, s=256, counts=256, T=4):
        return lib.moe_route_scores(256, B.MOE_F32, 64, bias, T, 64, 8, ops.route_rule(), ids, w, s, counts, None)
    for name in ("bias", "ids", "w", "s", "counts"):
        assert scores(**{name: bad}) == INVALID, name
    assert scores(counts=bad, T=0) == INVALID

    def backward(ids=256, dw=256, ds=256):
        return lib.moe_route_scores_backward(256, B.MOE_F32, 64, 4, 64, 8, ops.route_rule(), ids, dw, ds, 512, 64, None)
    for name in ("ids", "dw", "ds"):
        assert backward(**{name: bad}) == INVALID, name

    def combine(inv=256, w=256, dw=256):
        return lib.moe_combine_backward(256, 256, inv, w, 4, 2, 256, dw, 256, None)
    for name in ("inv", "w", "dw"):
        assert combine(**{name: bad}) == INVALID, name
    assert lib.moe_route_logits(256, 256, bad, 4, 128, 8, 256, None) == INVALID
    assert lib.moe_route_logits(256, 256, None, 4, 128, 8, bad, None) == INVALID


class Elsewhere(torch.Tensor):
    """A tensor without memory that says which device it is on."""
    __torch_dispatch__ = None


def refused_elsewhere():
    device = torch.device("cuda", torch.cuda.current_device() + 1 if torch.cuda.is_available() else 1)

    def new(*shape, dtype=torch.float32):
        return torch.Tensor._make_wrapper_subclass(Elsewhere, shape, dtype=dtype, device=device)
    rule, i32, bf16, u8 = ops.route_rule(), torch.int32, torch.bfloat16, torch.uint8
    op = object.__new__(ops.Nvfp4Operand)
    op.rows, op.K, op.device, op.struct = 128, 256, device.index, B.moe_nvfp4_operand(256, 256, 256, 1)
    op.q, op.s, op.gs = new(128 * 128, dtype=u8), new(2048, dtype=u8), new(128)
    ws = new(1 << 20, dtype=u8)
    calls = [lambda: ops.route_scores(new(4, 64), 8, rule),
             lambda: ops.route_scores_backward(new(4, 64), new(4, 8, dtype=i32), new(4, 8), rule),
             lambda: ops.combine_backward(new(4, 64, dtype=bf16), new(8, 64, dtype=bf16), new(8, dtype=i32), new(4, 2)),
             lambda: ops.nvfp4_quantize(new(128, 256), op),
             lambda: ops.nvfp4_matmul(op, op, torch.float32, ws),
             lambda: ops.nvfp4_linear(new(4, 256), op, ws)]
    if torch.cuda.is_available():  # (the Python-level checks ask torch for the current device)
        calls += [lambda: ops.route_logits(new(4, 128, dtype=bf16), new(8, 128)), op.values,
                  lambda: ops.nvfp4_workspace(4, 128, 256, device)]
    for call in calls:
        with pytest.raises(ValueError, match="another device than the current one"):
            call()


def test_tensors_of_another_device_are_refused():
    refused_elsewhere()


@pytest.mark.gpu
def test_tensors_of_another_device_are_refused_beside_a_gpu():
    refused_elsewhere()


@pytest.mark.gpu
def test_a_flag_without_a_truth_value_raises_its_own_error():
    two = torch.tensor([True, False])
    dy, w = torch.zeros(4, 64, device="cuda").bfloat16(), torch.zeros(4, 2, device="cuda")
    inv = torch.arange(8, dtype=torch.int32, device="cuda")
    with pytest.raises(RuntimeError, match="ambiguous"):
        ops.combine_backward(dy, dy.repeat(2, 1), inv, w, need_dw=two)
    with pytest.raises(RuntimeError, match="ambiguous"):
        ops.combine_backward(dy, dy.repeat(2, 1), inv, w, need_dy_perm=two)
    with pytest.raises(RuntimeError, match="ambiguous"):
        ops.nvfp4_quantize(dy, ops.nvfp4_operand(4, 64), scales_given=two)
