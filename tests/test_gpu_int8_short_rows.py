"""8-bit products of one step of 128 values a tile, several tiles a CTA: every other tile has no work for half of the converting warps."""
import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def whole(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("T,k,E,N,K", [(30, 32, 1024, 64, 64), (400, 32, 1024, 64, 64), (900, 4, 512, 130, 128), (3000, 8, 64, 300, 100), (500, 1, 300, 600, 1)])
def test_experts(T, k, E, N, K):
    g = gen(T)
    ids = R.some_ids(T, k, E, T, "distinct").cuda()
    x = torch.randn(T, K, generator=g, device="cuda")
    wq, s = whole(g, E, N, K), torch.rand(E, N, generator=g, device="cuda")
    W, ws = ops.int8_weights(wq, s), ops.int8_workspace(T * k, N, K)
    order = ops.expert_order(ids, E)
    rows = ops.int8_quantize(x, order)
    q, sx = R.numbers(x)
    want = torch.empty(T * k, N, device="cuda")
    flat = ids.view(-1).long()
    for pairs in torch.arange(T * k, device="cuda").split(4000):
        e, t = flat[pairs], pairs // k
        total = torch.einsum("pk,pnk->pn", q[t], wq[e].double())
        want[order.inv.view(-1)[pairs].long()] = total.float() * sx.float()[t][:, None] * s[e]
    for _ in range(60):
        assert torch.equal(ops.int8_matmul(rows, W, torch.float32, ws), want)
    assert B.moe_get_device_status(ws) == B.MOE_OK


@pytest.mark.parametrize("M,N,K", [(100, 60000, 128), (2000, 20000, 64), (5000, 9000, 127), (700, 40000, 1)])
def test_dense(M, N, K):
    g = gen(M)
    x, wq, s = torch.randn(M, K, generator=g, device="cuda").bfloat16(), whole(g, N, K), torch.rand(N, generator=g, device="cuda")
    W, ws = ops.int8_weights(wq, s), ops.int8_workspace(M, N, K)
    want = R.product(*R.numbers(x), wq, s, torch.bfloat16)
    for _ in range(40):
        assert torch.equal(ops.int8_linear(x, W, ws), want)
    assert B.moe_get_device_status(ws) == B.MOE_OK
