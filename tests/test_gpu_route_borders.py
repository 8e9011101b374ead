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
