"""Gradients of the weighted sum against 64 bits.  dw: an fp32 dot product whose longest serial chain has d/32 + 8 terms, then a
tree: (d/32 + 24) 2^-24 of the sum of the magnitudes.  dy_perm: one fp32 product rounded to bf16, equal bit for bit."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu


def inputs(T, k, d, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dy = torch.randn(T, d, generator=g, device="cuda").bfloat16()
    yp = torch.randn(T * k, d, generator=g, device="cuda").bfloat16()
    w = torch.randn(T, k, generator=g, device="cuda")
    inv = torch.randperm(T * k, generator=g, device="cuda").int()
    return dy, yp, inv, w


@pytest.mark.parametrize("T,k,d", [(1, 1, 8), (1, 8, 8192), (3, 5, 128), (9, 2, 264), (17, 9, 520), (5, 32, 1032),
                                   (333, 5, 2056), (2, 8, 16384), (1000, 1, 64), (64, 17, 4096)])
def test_gradients(T, k, d):
    dy, yp, inv, w = inputs(T, k, d)
    dw, dyp = ops.combine_backward(dy, yp, inv, w)
    rows = yp[inv.long()].double().view(T, k, d)
    prod = dy.double()[:, None, :] * rows
    err = (dw.double() - prod.sum(2)).abs()
    assert (err <= (d / 32 + 24) * 2.0 ** -24 * prod.abs().sum(2)).all()
    want = torch.empty_like(yp)
    want[inv.long()] = (w[:, :, None] * dy.float()[:, None, :]).bfloat16().view(T * k, d)
    assert torch.equal(dyp, want)
    dw1, none = ops.combine_backward(dy, yp, inv, w, need_dy_perm=False)
    none2, dyp1 = ops.combine_backward(dy, None, inv, w, need_dw=False)
    assert none is None and none2 is None and torch.equal(dw1, dw) and torch.equal(dyp1, dyp)


def test_entries_outside_the_rows():
    T, k, d = 4, 3, 64
    dy, yp, inv, w = inputs(T, k, d, 1)
    bad = inv.clone()
    bad[0], bad[4], bad[11] = -1, T * k, 2 ** 31 - 1
    dyp = torch.full_like(yp, 7.0)
    dw = torch.empty(T, k, device="cuda")
    from bit_expert_ffn_moe_gb300 import binding as B
    B.moe_combine_backward(dy, yp, bad, w, T, k, d, dw, dyp)
    whole, _ = ops.combine_backward(dy, yp, inv, w)
    flat, ref = dw.reshape(-1).cpu().numpy(), whole.reshape(-1).cpu().numpy()
    keep = np.ones(T * k, bool)
    keep[[0, 4, 11]] = False
    np.testing.assert_array_equal(flat[keep], ref[keep])
    assert (flat[~keep] == 0).all()
    untouched = inv.cpu()[[0, 4, 11]].long()
    assert (dyp[untouched] == 7.0).all()


def test_against_differences_of_the_weighted_sum():
    """dw is the derivative of <dy, y> for y of moe_combine's definition (linear in w: exact up to rounding)."""
    T, k, d = 6, 4, 256
    dy, yp, inv, w = inputs(T, k, d, 2)
    dw, _ = ops.combine_backward(dy, yp, inv, w)
    rows = yp.double()[inv.long()].view(T, k, d)

    def value(weights):
        return (dy.double() * (weights[:, :, None] * rows).sum(1)).sum(1)
    for j in range(k):
        h = torch.zeros(T, k, dtype=torch.float64, device="cuda")
        h[:, j] = 0.5
        diff = value(w.double() + h) - value(w.double() - h)
        assert (diff - dw[:, j].double()).abs().max() < 1e-3


def test_no_tokens():
    dw, dyp = ops.combine_backward(*inputs(0, 3, 64))
    assert dw.shape == (0, 3) and dyp.shape == (0, 64)
