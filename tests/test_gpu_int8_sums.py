"""Sums of the 8-bit products at 2^24 and beyond, in fp32, through every kernel: the dot products (up to 2 or 4 rows), a cluster's tiles, the
persistent kernel with single CTAs and with pairs, and by expert."""
import random

import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu
N = 24
ROWS = [1, 4, 40, 150, 700]
LIMIT = 2 ** 24


def products(q, w):
    """Name and result [.., N] in fp32 for scales of 1 of the row q, whose first number is 127, and the weights w [N, K]."""
    K = q.numel()
    W, twice = ops.int8_weights(w, torch.ones(N, device="cuda")), ops.int8_weights(w.expand(2, N, K).contiguous(), torch.ones(2, N, device="cuda"))
    for M in ROWS:
        x = q.float().expand(M, K).contiguous()
        yield "%d rows" % M, ops.int8_linear(x, W, ops.int8_workspace(M, N, K))
    for M in (10, 100):
        order = ops.expert_order((torch.arange(M, device="cuda") % 2).int()[:, None], 2)
        rows = ops.int8_quantize(q.float().expand(M, K).contiguous(), order)
        yield "%d by expert" % M, ops.int8_matmul(rows, twice, torch.float32, ops.int8_workspace(M, N, K))


def terms(K, choose):
    """The row q and the weights w [N, K] whose magnitudes are 90 .. 127 and whose signs choose(rng, sum so far, term, k) gives."""
    rng = random.Random(K)
    q, w = [127] + [rng.randint(90, 127) for _ in range(K - 1)], []
    for n in range(N):
        total, row = 0, []
        for k in range(K):
            m = rng.randint(100, 127)
            sign = choose(rng, total, q[k] * m, k)
            total += sign * q[k] * m
            row.append((sign if n % 2 else -sign) * m)
        w.append(row)
    q, w = torch.tensor(q, device="cuda"), torch.tensor(w, dtype=torch.int8, device="cuda")
    on_the_way = (q * w.long()).cumsum(1)
    return q, w, on_the_way[:, -1].double(), on_the_way.abs().amax(1).double()


@pytest.mark.parametrize("K", [1032, 4096, 20000])
def test_sums_that_stay_within_2_to_the_24_are_exact(K):
    """They come up to it and stay next to it."""
    q, w, want, most = terms(K, lambda rng, total, term, k: 1 if total + term <= LIMIT and (total < LIMIT - 40000 or rng.random() < 0.6) else -1)
    assert LIMIT - 400000 < int(most.max()) <= LIMIT if K > 2000 else int(most.max()) <= LIMIT
    for name, y in products(q, w):
        assert (y.double() == want).all(), name


@pytest.mark.parametrize("K", [8192, 32768])
@pytest.mark.parametrize("kind", ["cancel", "one sign"])
def test_sums_beyond(K, kind):
    """The dot products' are the exact sums rounded once; the tensor cores' are within K 2^-22 of the largest sum on the way: 16 products and
    a sum are 17 numbers, each cut off at 24 bits or more of the largest of them (2^-23), the result once more, K / 16 times; 18 / 16
    K 2^-23 is less.  Ranges of K that are joined add the rounding of a few additions, which the rest covers."""
    half = K // 2
    q, w, want, most = terms(K, lambda rng, total, term, k: 1 if k < half or kind == "one sign" else -1)
    assert (most > 2 * LIMIT).all()
    if kind == "cancel":
        assert (want.abs() < most / 50).all()
    for name, y in products(q, w):
        if name in ("1 rows", "10 by expert"):
            assert (y == want.float()).all(), name
        else:
            assert ((y.double() - want).abs() <= K * 2.0 ** -22 * most).all(), name
        assert (y == y[0]).all(), name
