"""8-bit products on the tensor cores whose CTAs compute whole tiles first and then share the last ones: single CTAs and pairs, of one matrix
and by expert, plain and gated, bit for bit.  shares() restates when tiles are shared, so that no case here is one of whole tiles alone."""
import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu
LEAST = 32  # steps of 128 values that sharing has to save, and that a share has


def shares(counts, N, K, pair, most):
    """Tiles that a CTA (or a pair) computes alone, and tiles that several share, for these rows of each expert."""
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    ctas = ctas // 2 if pair else ctas
    steps, tiles = -(-K // 128), sum(-(-c // most) for c in counts) * -(-N // (256 if pair else 128))
    rest = tiles % ctas
    sharers = min(ctas, max(rest, min(ctas, rest * steps // LEAST)))
    split = rest > 0 and steps - -(-rest * steps // sharers) >= LEAST
    return (tiles - rest, rest) if split else (tiles, 0)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def weights(g, *shape):
    return torch.randint(-40, 41, shape, generator=g, device="cuda", dtype=torch.int8)


def scales(g, *shape):
    return torch.rand(shape, generator=g, device="cuda") * 0.01 + 1e-4


def definition(q, s, wq, ws):
    return torch.cat([R.product(q, s, wq[n:n + 2000], ws[n:n + 2000], torch.float32) for n in range(0, len(wq), 2000)], 1)


@pytest.mark.parametrize("M,N,K", [(100, 30000, 12800), (17, 25001, 9000), (300, 25000, 12850), (1000, 4800, 9000), (2500, 5000, 16500)])
def test_one_matrix(M, N, K):
    """(Sums of K random terms of at most 127 x 40 are some 30 x 23 sqrt(K): they stay far below 2^24 on their way.)"""
    whole, shared = shares([M], N, K, M > 128, min(192, -(-M // 16) * 16))
    assert whole > 0 and shared > 0
    g = gen(M)
    x, wq, ws = torch.randn(M, K, generator=g, device="cuda").bfloat16(), weights(g, N, K), scales(g, N)
    W, space = ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K)
    want = definition(*R.numbers(x), wq, ws)
    for _ in range(3):
        assert torch.equal(ops.int8_linear(x, W, space), want.bfloat16())
    if N % 2 == 0:
        y, bound = R.gated_bound(want, torch.bfloat16)
        assert ((ops.int8_linear(x, W, space, gated=True).double() - y).abs() <= bound).all()
    assert B.moe_get_device_status(space) == B.MOE_OK


@pytest.mark.parametrize("counts,N,K", [([9, 0, 13, 11, 30, 3, 12, 8] * 6, 1000, 9100), ([1, 15] * 30, 380, 8500), ([0] * 20 + [10] * 60, 500, 20000),
                                        ([300, 17, 0, 64, 128, 129, 1, 500], 2600, 9000), ([40] * 30, 1500, 12800)])
def test_by_expert(counts, N, K):
    E, M = len(counts), sum(counts)
    mean = M // E
    most = min(192, -(-min(M, mean + (3 * mean + 16 if mean < 16 else 64)) // 16) * 16)
    whole, shared = shares(counts, N, K, mean >= 16, most)
    assert whole > 0 and shared > 0
    g = gen(M)
    ids = torch.cat([torch.full((c,), e, dtype=torch.int32) for e, c in enumerate(counts)])
    ids = ids[torch.randperm(M, generator=torch.Generator().manual_seed(M))].cuda()
    order = ops.expert_order(ids[:, None], E)
    x, wq, ws = torch.randn(M, K, generator=g, device="cuda").half(), weights(g, E, N, K), scales(g, E, N)
    W, space = ops.int8_weights(wq, ws), ops.int8_workspace(M, N, K)
    q, s = R.numbers(x)
    want = torch.empty(M, N, device="cuda")
    for e in range(E):
        t = torch.nonzero(ids == e)[:, 0]
        if len(t):
            want[order.inv[t, 0].long()] = definition(q[t], s[t], wq[e], ws[e])
    rows = ops.int8_quantize(x, order)
    for _ in range(3):
        assert torch.equal(ops.int8_matmul(rows, W, torch.float32, space), want)
    y, bound = R.gated_bound(want, torch.float16)
    assert ((ops.int8_matmul(rows, W, torch.float16, space, gated=True).double() - y).abs() <= bound).all()
    assert B.moe_get_device_status(space) == B.MOE_OK
