"""Sizes at which the weighted sum's gradients and the row operands take another of their variants.  Tolerance of dw: as in the other tests
of these gradients, (d/32 + 24) 2^-24 of the sum of the magnitudes; dy_perm is one rounding, equal bit for bit."""
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu


# one slot: rows of more pieces than the CTA's threads take at once, and whole / half / odd numbers of turns; two to four slots: two pieces at a
# time, the last turn of one; five to eight: one piece, 257 .. 320 of them by 320 threads, 513 by 256; more: even turns of each number of slots
@pytest.mark.parametrize("T,k,d", [(7, 1, 8200), (3, 1, 16392), (5, 1, 32768), (9, 1, 2048), (6, 2, 4104), (4, 2, 8192), (5, 2, 4112), (6, 3, 4104),
                                   (3, 3, 8216), (6, 4, 4104), (2, 4, 16392), (5, 5, 2560), (5, 6, 2304), (7, 7, 2056), (4, 7, 4104), (3, 8, 4104),
                                   (4, 9, 2560), (3, 13, 2056), (2, 14, 4104), (2, 21, 1032), (2, 31, 2304)])
def test_gradients_of_the_weighted_sum(T, k, d):
    g = torch.Generator(device="cuda").manual_seed(T * k + d)
    dy = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    yp = torch.randn(T * k, d, generator=g, device="cuda").bfloat16()
    w = torch.randn(T, k, generator=g, device="cuda")
    inv = torch.randperm(T * k, generator=g, device="cuda").int()
    dw, dyp = ops.combine_backward(dy, yp, inv, w)
    prod = dy.double()[:, None, :] * yp[inv.long()].double().view(T, k, d)
    assert ((dw.double() - prod.sum(2)).abs() <= (d / 32 + 24) * 2.0 ** -24 * prod.abs().sum(2)).all()
    want = torch.empty_like(yp)
    want[inv.long()] = (w[:, :, None] * dy.float()[:, None, :]).bfloat16().view(T * k, d)
    assert torch.equal(dyp, want)
    dw1, _ = ops.combine_backward(dy, yp, inv, w, need_dy_perm=False)
    _, dyp1 = ops.combine_backward(dy, None, inv, w, need_dw=False)
    assert torch.equal(dw1, dw) and torch.equal(dyp1, dyp)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K", [40, 1024, 8191, 8192, 9000])
def test_a_rows_operand_does_not_depend_on_its_batch(dtype, K):
    """Codes and scales of the same rows alone, in a small batch and in one that is streamed: the same values and row scales, bit for bit."""
    x = torch.randn(2600, K, generator=torch.Generator(device="cuda").manual_seed(K), device="cuda").to(dtype)
    whole = ops.nvfp4_operand(2600, K)
    ops.nvfp4_quantize(x, whole)
    values = whole.values()
    for first, n in ((0, 1), (77, 16), (128, 300), (2599, 1)):
        part = ops.nvfp4_operand(n, K)
        ops.nvfp4_quantize(x[first:first + n], part)
        assert torch.equal(part.gs, whole.gs[first:first + n])
        assert torch.equal(part.values(), values[first:first + n])
