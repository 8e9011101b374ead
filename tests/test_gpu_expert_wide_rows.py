"""Rows between tokens and experts of nearly 2^31 elements: every element, and weights' gradients of sums that are exact."""
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu


def equal(a, b, f):
    """Whether a is f of b, 2^27 elements at a time."""
    return all(torch.equal(a[i:i + 2 ** 27], f(b[i:i + 2 ** 27])) for i in range(0, a.numel(), 2 ** 27))


@pytest.mark.parametrize("d", [2 ** 31 - 8, 2 ** 31 - 1])  # pieces of 16 bytes, words
def test_rows_of_nearly_2_to_the_31_elements(d):
    """One token of one slot: `rows` of -1, 0 and 1, `x` of -1 and 1 at the ends and some places between, so that the sum for the weight's
    gradient has some 40000 whole numbers."""
    g = torch.Generator(device="cuda").manual_seed(d % 97)
    x, rows = torch.zeros(1, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    for i in range(0, d, 2 ** 27):
        rows[0, i:i + 2 ** 27] = torch.randint(-1, 2, (min(2 ** 27, d - i),), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    some = torch.cat((torch.arange(0, 9000, device="cuda"), torch.arange(d - 20000, d, device="cuda"),
                      torch.randint(0, d, (10000,), generator=g, device="cuda").unique())).unique()
    x[0, some] = (2 * torch.randint(0, 2, (len(some),), generator=g, device="cuda") - 1).bfloat16()
    want = float((x[0, some].double() * rows[0, some].double()).sum())
    order = ops.expert_order(torch.zeros(1, 1, dtype=torch.int32, device="cuda"), 1)
    w = torch.full((1, 1), 0.5, device="cuda")
    dx, dw = ops.tokens_to_experts_backward(rows, order, x, w)
    assert float(dw) == want and equal(dx[0], rows[0], lambda r: 0.5 * r)
    del dx
    drows, dw = ops.experts_to_tokens_backward(x, order, rows, w)
    assert float(dw) == want and equal(drows[0], x[0], lambda r: 0.5 * r)
    del drows
    for y, of in ((ops.tokens_to_experts(rows, order), rows), (ops.experts_to_tokens(rows, order), rows)):
        assert equal(y[0], of[0], lambda r: r)
