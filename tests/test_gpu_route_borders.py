"""The routing rules where the ranking values leave fp32's reach: infinite, NaN and very large bias values, groups whose two best values
cancel.  Against a 64-bit choice written out here; ids have to be equal.  Weights: as many roundings as in the other tests of the
rules, 2^-17 of softmax and 2^-19 of sigmoid."""
import numpy as np
import pytest
import torch

from bit_expert_ffn_moe_gb300 import ops

pytestmark = pytest.mark.gpu


def choose(logits, bias, k, score, groups, top_groups, group_score):
    """ids [T][k] and scores [T][E] in fp64: infinite bias values rank first and last, NaN ones with the experts out of service; neither of
    the latter two counts in a group's score."""
    l, b = np.asarray(logits, np.float64), np.asarray(bias, np.float64)
    T, E = l.shape
    of = np.arange(E) // (E // groups)
    ids, scores = np.zeros((T, k), np.int32), np.zeros((T, E))
    for t in range(T):
        served = l[t] > -np.inf
        if score == "sigmoid":
            s = np.where(served, 1.0 / (1.0 + np.exp(-np.where(served, l[t], 0.0))), 0.0)
        else:
            p = np.where(served, np.exp(np.where(served, l[t] - l[t][served].max(initial=-1e300), 0.0)), 0.0)
            s = p / p.sum() if served.any() else p
        v = s + b
        ranked = served & ~np.isnan(v)
        best = np.full(groups, -np.inf)
        for g in range(groups):
            vals = np.sort(v[ranked & (of == g) & (v > -np.inf)])[::-1]
            if len(vals):
                best[g] = vals[0] if group_score == "max" or np.isinf(vals[0]) else vals[:2].sum()
        kept = np.argsort(-best, kind="stable")[:top_groups]
        cand = [e for e in range(E) if of[e] in kept]
        cand.sort(key=lambda e: (0, -v[e], e) if ranked[e] else (1, 0.0, e))
        ids[t], scores[t] = sorted(cand[:k]), s
    return ids, scores


def check(logits, bias, k, score, groups=1, top_groups=1, group_score="top2"):
    E = logits.shape[1]
    bias = np.asarray(bias, np.float32)
    rule = ops.route_rule(score, groups, top_groups, group_score)
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    ids, w = ops.route_scores(torch.from_numpy(logits).cuda(), k, rule, torch.from_numpy(bias).cuda(), counts=counts)
    ref, s = choose(logits, bias, k, score, groups, top_groups, group_score)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref)
    np.testing.assert_array_equal(counts.cpu().numpy(), np.bincount(ref.reshape(-1), minlength=E))
    u = np.take_along_axis(s, ref, 1)
    S = u.sum(1, keepdims=True)
    want = np.where(S > 0, u / np.where(S > 0, S, 1.0), 0.0)
    np.testing.assert_allclose(w.double().cpu().numpy(), want, rtol=2.0 ** -17 if score == "softmax" else 2.0 ** -19, atol=1e-37)


RULES = [(1, 1, "max"), (8, 3, "max"), (8, 3, "top2"), (20, 7, "top2"), (32, 4, "top2")]


def widths(groups):
    return (64, 256) if 64 % groups == 0 else (80, 100)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups,group_score", RULES)
@pytest.mark.parametrize("pins", [1, 2, 5, 40])
def test_a_bias_of_inf_picks_first(score, groups, top_groups, group_score, pins):
    rng = np.random.default_rng(pins + groups)
    for E in widths(groups):
        for k in (1, 4, min(20, top_groups * (E // groups))):
            if k > top_groups * (E // groups):
                continue
            l = rng.standard_normal((33, E)).astype(np.float32)
            l[3] = -np.inf
            l[4, ::2] = -np.inf
            l[5, 1:] = np.nan
            bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
            bias[rng.permutation(E)[:pins]] = np.inf
            check(l, bias, k, score, groups, top_groups, group_score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("groups,top_groups,group_score", RULES)
@pytest.mark.parametrize("seed", range(4))
def test_bias_values_of_every_kind(score, groups, top_groups, group_score, seed):
    """+-inf, NaN, the largest and the lowest finite number among ordinary ones, from a few of them to nothing else."""
    rng = np.random.default_rng(seed)
    kinds = np.array([np.inf, -np.inf, np.nan, 3.4028234e38, -3.4028234e38, 1e9, 0.0, 0.25], np.float32)
    for E in widths(groups):
        for share in (0.1, 0.5, 1.0):
            for k in (1, 3, min(9, top_groups * (E // groups))):
                l = rng.standard_normal((17, E)).astype(np.float32)
                l[2, :E // 2] = -np.inf
                bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
                odd = rng.random(E) < share
                bias[odd] = kinds[rng.integers(0, len(kinds), int(odd.sum()))]
                check(l, bias, min(k, top_groups * (E // groups)), score, groups, top_groups, group_score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top_groups", [(64, 32, 5), (96, 32, 5), (100, 20, 7), (256, 32, 3), (64, 8, 3)])
@pytest.mark.parametrize("size", [10.0, 1000.0, 1e5])
def test_groups_whose_best_two_cancel(score, E, groups, top_groups, size):
    """Bias values of opposite sign in each group: the sum of its two best is a thousandth of either, and fp32 knows it to the rounding of
    those."""
    rng = np.random.default_rng(int(size) + E)
    l = (1e-3 * rng.standard_normal((300, E))).astype(np.float32)
    bias = np.full(E, -size, np.float32)
    bias[::E // groups] = size
    for k in (1, top_groups):
        check(l, bias, k, score, groups, top_groups, "top2")
    bias += (1e-4 * rng.standard_normal(E)).astype(np.float32)
    check(l, bias, 2, score, groups, top_groups, "top2")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,top_groups", [(64, 32, 20), (96, 32, 20), (100, 20, 15), (64, 8, 6)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups_of_the_lowest_bias_rank_before_groups_out_of_service(score, E, groups, top_groups, group_score):
    """The type's lowest number as the bias that switches experts off: two of them add up below fp32's range."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((64, E)).astype(np.float32)
    per = E // groups
    bias = np.zeros(E, np.float32)
    bias[3 * per:] = np.finfo(np.float32).min
    for t in range(64):
        for g in rng.permutation(groups)[:groups - top_groups + rng.integers(-2, 3)]:
            l[t, g * per:(g + 1) * per] = -np.inf
    for k in (1, 5, min(30, top_groups * per)):
        check(l, bias, k, score, groups, top_groups, group_score)
