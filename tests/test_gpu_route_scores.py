"""Routing rules and their gradient on the GPU against the 64-bit forms: ids equal, weights and gradients within the roundings of
the fp32 formulas.

Tolerances.  A score costs exp, a sum and a division in fp32: at most 4 roundings (2^-24 each, exp two of them) and, for
softmax, the sum's E/32 + 5 and the argument's |l - max|; a renormalised weight adds the sum over the picks.  With
E <= 1024 and |l - max| <= 32 these stay below 2^-17 for softmax and 2^-19 for sigmoid, relative.  A gradient is a sum of such
terms: 2^-16 of the sum of their magnitudes (row sums included), plus half a step of its type."""
import numpy as np
import pytest
import torch

import ops_reference as R
from bit_expert_ffn_moe_gb300 import binding as B
from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in TYPES.values()}


def check(logits, k, bias=None, score="sigmoid", groups=1, top_groups=1, group_score="top2", renormalize=True, scale=1.0,
          backward=True, stride=None):
    """logits: CPU tensor of any of the types."""
    T, E = logits.shape
    dev = logits.cuda()
    if stride is not None:
        room = torch.full((T, stride), float("nan"), dtype=logits.dtype, device="cuda")
        room[:, :E] = dev
        dev = room[:, :E]
    rule = ops.route_rule(score, groups, top_groups, group_score, renormalize, scale)
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32).cuda()
    scores = torch.empty(T, E, device="cuda")
    counts = torch.full((E,), 77, dtype=torch.int32, device="cuda")
    ids, w = ops.route_scores(dev, k, rule, b, scores, counts)
    l64 = logits.double().numpy()
    bias64 = None if b is None else b.double().cpu().numpy()
    ids_r, w_r, s_r = R.route(l64, k, bias64, score, groups, top_groups, group_score, renormalize, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), ids_r)
    rtol = 2.0 ** -17 if score == "softmax" else 2.0 ** -19
    np.testing.assert_allclose(w.double().cpu().numpy(), w_r, rtol=rtol, atol=1e-37)
    np.testing.assert_allclose(scores.double().cpu().numpy(), s_r, rtol=rtol, atol=1e-37)
    np.testing.assert_array_equal(counts.cpu().numpy(), np.bincount(ids_r.reshape(-1), minlength=E))
    ids2, w2 = ops.route_scores(dev, k, rule, b)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    if not backward:
        return ids_r, w_r
    rng = np.random.default_rng(E + k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    for dscores in (None, rng.standard_normal((T, E)).astype(np.float32)):
        ds = None if dscores is None else torch.from_numpy(dscores).cuda()
        dl = ops.route_scores_backward(dev, ids, torch.from_numpy(dw).cuda(), rule, ds)
        assert dl.dtype == logits.dtype
        ref, mag = R.route_backward(l64, ids_r, dw, score, renormalize, scale, dscores)
        err = np.abs(dl.double().cpu().numpy() - ref)
        tol = 2.0 ** -16 * mag + HALF_STEP[logits.dtype] * np.abs(ref) + (6e-8 if logits.dtype == torch.float16 else 1e-37)
        assert (err <= tol).all(), float((err - tol).max())
    return ids_r, w_r


def randn(T, E, seed, dtype="fp32", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * scale).to(TYPES[dtype])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,group_score,biased,renorm,scale", [
    (1, 256, 8, 8, 4, "top2", True, True, 2.5),
    (37, 128, 8, 1, 1, "top2", False, True, 1.0),
    (5, 1, 1, 1, 1, "max", True, True, 1.0),
    (9, 31, 31, 1, 1, "max", True, False, 1.0),
    (11, 33, 5, 3, 2, "top2", False, True, 1.0),
    (13, 160, 6, 8, 3, "max", True, False, 16.0),
    (8, 1000, 32, 20, 7, "top2", True, True, 2.5),
    (3, 1024, 17, 32, 32, "max", True, True, 1.0),
    (6, 96, 4, 32, 5, "top2", True, True, 1.0),   # three experts per group
    (6, 32, 2, 32, 2, "top2", True, True, 1.0),   # one per group: a sum of one
])
def test_rules(dtype, score, T, E, k, groups, top_groups, group_score, biased, renorm, scale):
    bias = None
    if biased:
        bias = torch.randn(E, generator=torch.Generator().manual_seed(5)) * (0.1 if score == "sigmoid" else 0.5 / E)
    check(randn(T, E, 7 * E + k, dtype), k, bias, score, groups, top_groups, group_score, renorm, scale)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups,group_score", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_id(score, groups, top_groups, group_score, biased):
    """Whole-number logits and bias values from a grid of a few: exact ties at the border of the choice in most rows."""
    rng = np.random.default_rng(1)
    l = torch.from_numpy(rng.integers(-2, 3, size=(40, 64)).astype(np.float32))
    l[0] = 0.0
    bias = rng.integers(0, 2, size=64).astype(np.float32) * 0.25 if biased else None
    check(l, 7, bias, score, groups, top_groups, group_score)
    check(l, 7, None if bias is None else 0 * bias, score, groups, top_groups, group_score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_near_ties_are_decided_as_in_64_bits(score):
    """Bias values that bring pairs of experts within a few 2^-26 of one another, on both sides: fp32 cannot order them."""
    rng = np.random.default_rng(2)
    T, E, k = 64, 64, 8
    l = rng.standard_normal((T, E)).astype(np.float32)
    s = R.route(l[:1], k, score=score)[2][0]
    bias = (1.0 - s).astype(np.float32)          # row 0: every value is 1 up to the bias's rounding
    order = rng.permutation(E)
    bias[order[:16]] += np.float32(2.0 ** -24)
    l[1:] = l[0] + rng.integers(-1, 2, size=(T - 1, E)).astype(np.float32) * 1e-6
    check(torch.from_numpy(l), k, bias, score)
    check(torch.from_numpy(l), k, bias, score, groups=8, top_groups=3)
    check(torch.from_numpy(l), k, bias, score, groups=8, top_groups=3, group_score="max")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups,top_groups,group_score", [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2")])
def test_experts_out_of_service(score, biased, groups, top_groups, group_score):
    """-inf and NaN logits, rows with fewer than k experts left, one left, none left; a bias does not bring them back."""
    T, E, k = 24, 64, 6
    l = randn(T, E, 11)
    l[:, 5] = -float("inf")
    l[1] = -float("inf")
    l[2] = float("nan")
    l[3] = -float("inf")
    l[3, 40] = 0.5
    l[4, 8:] = -float("inf")
    l[5, ::2] = -float("inf")
    l[6, 10:20] = float("nan")
    l[7, :8] = torch.finfo(torch.float32).min  # the type's lowest value is in service
    bias = np.linspace(-1, 1, E).astype(np.float32) if biased else None
    if bias is not None:
        bias[5] = 100.0
    ids, w = check(l, k, bias, score, groups, top_groups, group_score, backward=False)
    np.testing.assert_array_equal(ids[1], np.arange(k))
    assert (w[1] == 0).all() and (w[2] == 0).all() and w[3].sum() == pytest.approx(1.0)
    rule = ops.route_rule(score, groups, top_groups, group_score)
    ids_d = torch.from_numpy(ids).cuda()
    dl = ops.route_scores_backward(l.cuda(), ids_d, torch.ones(T, k, device="cuda"), rule)
    assert torch.isfinite(dl).all() and (dl[1] == 0).all() and (dl[:, 5] == 0).all()


def test_extreme_logits():
    """Scores that saturate, underflow or sit at the ends of the range keep their order and ratios."""
    l = torch.zeros(8, 64)
    l[0] = torch.linspace(-120, -60, 64)
    l[1] = torch.linspace(60, 120, 64)
    l[2] = -100.0
    l[3, ::3] = 3e38
    l[4] = torch.linspace(-1e38, 1e38, 64)
    l[5, 7] = float("inf")
    l[5, 9] = float("inf")
    l[6] = -3e38
    l[7] = torch.linspace(-30, 30, 64)
    for renorm in (True, False):
        rule = ops.route_rule("sigmoid", renormalize=renorm)
        ids, w = ops.route_scores(l.cuda(), 4, rule)
        ids_r, w_r, _ = R.route(l.numpy(), 4, renormalize=renorm)
        np.testing.assert_array_equal(ids.cpu().numpy(), ids_r)
        np.testing.assert_allclose(w.double().cpu().numpy(), w_r, rtol=2.0 ** -17, atol=1e-37)
        rule = ops.route_rule("softmax", renormalize=renorm)
        ids, w = ops.route_scores(l.cuda(), 4, rule)
        ids_r, w_r, _ = R.route(l.numpy(), 4, score="softmax", renormalize=renorm)
        np.testing.assert_array_equal(ids.cpu().numpy(), ids_r)
        np.testing.assert_allclose(w.double().cpu().numpy(), w_r, rtol=2.0 ** -16, atol=1e-37)


@pytest.mark.parametrize("dtype,stride", [("fp32", 257), ("bf16", 131), ("fp16", 1000)])
def test_strided_rows(dtype, stride):
    check(randn(10, 130, 4, dtype), 5, torch.linspace(-.1, .1, 130), groups=2, top_groups=1, stride=stride)


def test_no_rows_and_other_streams():
    rule = ops.route_rule()
    counts = torch.full((64,), 9, dtype=torch.int32, device="cuda")
    ids, w = ops.route_scores(torch.empty(0, 64, device="cuda"), 4, rule, counts=counts)
    assert ids.shape == (0, 4) and int(counts.sum()) == 0
    l = randn(300, 64, 8).cuda()
    want = ops.route_scores(l, 4, rule)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops.route_scores(l, 4, rule)
        dl = ops.route_scores_backward(l, got[0], got[1], rule)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert torch.equal(dl, ops.route_scores_backward(l, want[0], want[1], rule))


def test_ids_outside_the_experts_take_no_part():
    l = randn(4, 64, 9).cuda()
    rule = ops.route_rule(renormalize=False)
    ids = torch.tensor([[1, 64], [-1, 2], [3, 1 << 30], [4, 5]], dtype=torch.int32, device="cuda")
    dl = ops.route_scores_backward(l, ids, torch.ones(4, 2, device="cuda"), rule).cpu()
    assert [int((r != 0).sum()) for r in dl] == [1, 1, 1, 2]


def test_logits_call_feeds_the_rules():
    """The exposed logits are moe_route's: the plain softmax rule on them chooses and weighs as moe_route does."""
    from bit_expert_ffn_moe_gb300 import inputs as IN
    from bit_expert_ffn_moe_gb300.layer import make_workspace
    from moe_testlib import bits_to_device
    cfg = IN.CONFIGS["tiny"]
    x = bits_to_device(IN.make_x(cfg)).view(torch.bfloat16)
    W_r, b = (torch.from_numpy(v).cuda() for v in IN.make_router(cfg))
    ids, w = ops.route_scores(ops.route_logits(x, W_r, b), cfg.k, ops.route_rule("softmax"))
    ws = make_workspace(cfg.T, cfg.d, cfg.E, cfg.k, cfg.I, B.MOE_ACT_BF16)
    ids0, w0 = torch.empty_like(ids), torch.empty_like(w)
    B.moe_route(x, W_r, b, cfg.T, cfg.d, cfg.E, cfg.k, ids0, w0, ws)
    assert torch.equal(ids, ids0)
    np.testing.assert_allclose(w.cpu().numpy(), w0.cpu().numpy(), rtol=2.0 ** -19)


@pytest.mark.parametrize("T,E,k", [(1, 7, 1), (3, 33, 3), (67, 1000, 32), (130, 64, 5), (1001, 300, 17)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_sparse_gradient_equals_the_dense_one(score, T, E, k):
    """A gradient of the scores of zero asks for the dense kernel: it rounds the same products, of a softmax with one subtraction of a
    sum that is zero but for its roundings (k products, each off by 2^-24 of itself or less, and k sums)."""
    g = torch.Generator().manual_seed(T + E)
    logits = (3 * torch.randn(T, E + 5, generator=g)).cuda()[:, 2:2 + E]
    dw = torch.randn(T, k, generator=g).cuda()
    rule = ops.route_rule(score, scale=1.5)
    ids, _ = ops.route_scores(logits, k, rule)
    sparse = ops.route_scores_backward(logits, ids, dw, rule)
    dense = ops.route_scores_backward(logits, ids, dw, rule, torch.zeros(T, E, device="cuda"))
    bound = 1.5 * dw.abs().sum(1, keepdim=True) * (4 * k + 16) * 2.0 ** -24
    assert ((sparse - dense).abs() <= bound).all()
    assert (sparse.gather(1, ids.long()) != 0).any() or k == 1
