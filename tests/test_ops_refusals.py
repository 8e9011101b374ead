"""Refusals of the routing rules, the weighted sum's gradients and the NVFP4 products beyond those of null pointers and shapes."""
import pytest

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
