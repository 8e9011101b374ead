"""A wait that runs out where the copying thread has issued everything already: its copies land before the CTA's shared memory is looked
at or goes (the self-test reports another status if they have not), and the 8-bit products run as before afterwards."""
import expert_reference as R
import pytest
import torch

from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit_us", [1, 5, 2000])
def test_copies_land_where_another_threads_wait_runs_out(limit_us):
    g = torch.Generator(device="cuda").manual_seed(limit_us)
    M, N, K = 150, 300, 700
    x = torch.randn(M, K, generator=g, device="cuda")
    wq = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    W, ws = ops.int8_weights(wq, torch.ones(N, device="cuda")), ops.int8_workspace(M, N, K)
    want = R.product(*R.numbers(x), wq, torch.ones(N, device="cuda"), torch.float32)
    for _ in range(20):
        B.moe_selftest_wait_timeout(ws, limit_us)
        assert B.moe_get_device_status(ws) == B.MOE_ERR_TIMEOUT
    assert torch.equal(ops.int8_linear(x, W, ws), want) and B.moe_get_device_status(ws) == B.MOE_OK
