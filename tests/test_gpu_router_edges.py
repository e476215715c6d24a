"""moe_router_topk where fp32 underflows, where choices lie closer than its error, and with infinite biases, against
the float64 oracle.

Chosen experts must be equal.  A weight is a score, over the sum of up to 64 of them if asked, times scale.  Roundings
of 2^-24 relative on its way: the exponential's argument, rounded to fp32 (a softmax's is a difference of up to twice
the row's reach |x|): 2 reach; the exponential itself 2; a softmax's sum of up to 16 terms a lane and 6 levels of
lanes, or 32 and 4, of terms with 4 each: 40; quotients, products, the sum of the chosen: 20.  Weights that fp32 holds
as subnormals are rounded to its smallest step, 2^-149.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_moe_amd as fm
from oracle.router import router_reference
from tests.gpu_helpers import say

pytestmark = pytest.mark.gpu

SCORES = {"softmax": fm.SCORE_SOFTMAX, "sigmoid": fm.SCORE_SIGMOID}
INF, NAN = float("inf"), float("nan")


def check(logits, K, score, bias=None, rows=slice(None), **kw):
    ids, w = fm.moe_router_topk(logits.cuda(), K, SCORES[score], bias=None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy()[rows], w.cpu().double().numpy()[rows]
    x = logits.double().numpy()[rows]
    rid, rw = router_reference(x, K, score, None if bias is None else bias.double().numpy(), **kw)
    assert np.array_equal(ids, rid), f"rows {np.flatnonzero((ids != rid).any(1))[:8]}"
    reach = np.abs(np.where(np.isfinite(x), x, 0.0)).max(1) * (2 if score == "softmax" else 1)
    assert np.all(np.abs(w - rw) <= np.abs(rw) * ((2 * reach + 64) * 2.0 ** -24)[:, None] + 2.0 ** -149)
    return ids, w


@pytest.mark.parametrize("E,K", [(8, 4), (128, 8), (512, 8), (1024, 20)])
@pytest.mark.parametrize("at", [-60.0, -70.0, -86.0, -87.5, -89.0, -100.0, -600.0])
def test_sigmoid_scores_that_underflow_in_fp32(E, K, at):
    say("router far sigmoid", E, K, at)
    g = torch.Generator().manual_seed(E)
    logits = at + torch.randn(9, E, generator=g)
    bias = 0.1 * torch.randn(E, generator=g)
    for renormalize in (True, False):
        for b in (None, bias):
            _, w = check(logits, K, "sigmoid", b, renormalize=renormalize)
            if renormalize:
                assert np.allclose(w.sum(1), 1.0, rtol=1e-4)
    check(logits, K, "sigmoid", bias, renormalize=False, scale=2.0 ** 100)
    check(logits, K, "sigmoid", n_group=4, topk_group=2, group_top=2)
    check(logits.bfloat16(), K, "sigmoid", n_group=4, topk_group=2)


@pytest.mark.parametrize("E,K", [(8, 4), (128, 8), (512, 8), (1024, 20)])
@pytest.mark.parametrize("below", [60.0, 80.0, 100.0, 110.0, 500.0])
def test_softmax_scores_that_underflow_in_fp32(E, K, below):
    """The row's largest logit belongs to an expert that its bias, or its group's, rules out."""
    say("router far softmax", E, K, below)
    g = torch.Generator().manual_seed(E + 1)
    logits = torch.randn(9, E, generator=g)
    logits[:, 2] += below
    bias = torch.zeros(E)
    bias[2] = -INF
    _, w = check(logits, K, "softmax", bias)
    assert np.allclose(w.sum(1), 1.0, rtol=1e-4)
    check(logits, K, "softmax", bias, renormalize=False, scale=2.0 ** 100)
    per = E // 4
    bias = torch.zeros(E)
    bias[:per] = -1.0
    bias[2] = -3.0
    check(logits, min(K, per), "softmax", bias, n_group=4, topk_group=1)
    # chosen beside the largest: a weight of its own, however small
    check(logits, K, "softmax", renormalize=False, scale=2.0 ** 100)
    check(logits, K, "softmax", scale=2.0 ** 100)


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("E,n_group", [(16, 4), (256, 8), (60, 4)])
def test_infinite_biases_in_groups(score, E, n_group):
    """A group whose only expert left has the bias +inf counts as -inf where two choices are asked of it."""
    say("router infinite biases", score, E, n_group)
    per = E // n_group
    g = torch.Generator().manual_seed(E)
    logits = torch.randn(20, E, generator=g)
    bias = 0.1 * torch.randn(E, generator=g)
    last = (n_group - 1) * per
    bias[last + 1] = INF
    logits[:, last:] = -INF
    logits[:, last + 1] = torch.randn(20, generator=g)
    K = min(8, per)
    ids, _ = check(logits, K, score, bias, n_group=n_group, topk_group=2, group_top=2)
    assert not (ids >= last).any()
    for top in (1, 2):      # two infinite choices, and one of each sign
        logits[:, last] = 0.5
        check(logits, K, score, bias, n_group=n_group, topk_group=2, group_top=top)
        bias[last] = INF
        check(logits, K, score, bias, n_group=n_group, topk_group=2, group_top=top)
        bias[0] = -INF
        check(logits, K, score, bias, n_group=n_group, topk_group=1, group_top=top)
        bias[0] = 3.4e38
        bias[1] = 3.4e38    # a sum beyond fp32
        check(logits, K, score, bias, n_group=n_group, topk_group=2, group_top=top)


# m, a, b, c: s(a) + s(b) exceeds 2 s(c) by less than 2^-23 of it, where s(v) = exp(v - m); the fp32 roundings of
# the differences from m and of the exponentials' arguments add up to 100 of those steps the other way
FAR = [(32.300010681152344, -32.12515640258789, -32.02237319946289, -32.072444915771484),
       (32.099998474121094, -32.00337600708008, -32.10615921020508, -32.05344772338867),
       (32.400001525878906, -32.25282669067383, -32.35560989379883, -32.30289840698242),
       (32.400001525878906, -32.345890045166016, -32.448673248291016, -32.39596176147461)]


@pytest.mark.parametrize("m,a,b,c", FAR)
def test_close_groups_far_below_the_largest_logit(m, a, b, c):
    """Groups by sums of scores so small that their roundings exceed a fixed multiple of fp32's step."""
    say("router far groups", m, a, b, c)
    rows = torch.tensor([[m, m, a, b, c, c, -INF, -INF], [m, m, c, c, a, b, -INF, -INF]])
    s = lambda v: np.exp(np.float64(v) - m)
    assert 0 < (s(a) + s(b)) / (2 * s(c)) - 1 < 2.0 ** -23
    ids, _ = check(rows, 4, "softmax", n_group=4, topk_group=2, group_top=2)
    assert sorted(ids[0].tolist()) == [0, 1, 2, 3] and sorted(ids[1].tolist()) == [0, 1, 4, 5]


@pytest.mark.parametrize("m", [32.4, 33.0])
def test_biases_of_the_size_of_far_scores(m):
    """Softmax scores of 2^-93 and biases of that size: the larger score's rounding up and the smaller's down must not
    decide."""
    f = np.float32
    m = f(m)
    v = np.unique(-(f(31.7) + np.random.default_rng(3).random(200000).astype(f)))
    a = ((v - m) * f(1.4426950408889634)).astype(np.float64)      # the exponential's argument in fp32
    true = np.exp(v.astype(np.float64) - np.float64(m))
    err = np.exp2(a) / true - 1
    v1, v2 = np.argmax(err), np.argmin(err)
    assert err[v1] - err[v2] > 90 * 2.0 ** -23
    b2 = f((true[v1] - true[v2]) + 3 * 2.0 ** -23 * true[v1])      # expert 2 leads by three steps
    assert 0 < true[v2] + np.float64(b2) - true[v1] < 5 * 2.0 ** -23 * true[v1]
    logits = torch.tensor([[m, v[v1], v[v2]] + [-200.0] * 5])
    bias = torch.zeros(8)
    bias[2] = float(b2)
    say("router far biases", m, v[v1], v[v2], b2)
    ids, _ = check(logits, 3, "softmax", bias)
    assert ids[0].tolist() == [0, 2, 1]


def test_biases_of_the_size_of_subnormal_scores():
    """A score below fp32's smallest normal value against a bias just below it."""
    logits = torch.tensor([[0.0, -88.0, -100.0] + [-200.0] * 5])
    bias = torch.zeros(8)
    bias[2] = 5e-39
    ids, _ = check(logits, 3, "softmax", bias)
    assert ids[0].tolist() == [0, 1, 2]


def test_a_later_choice_of_a_larger_error():
    """Softmax, one slot: two choices of tiny scores, further apart than their errors, stand ahead of one whose score is
    near 1 and whose fp32 value is too low by more than what parts it from them."""
    f = np.float32
    low = -np.random.default_rng(5).uniform(3.5, 4.5, 20000).astype(f)
    z = 1 + np.exp(low.astype(np.float64))
    z32 = z.astype(f)
    s32 = (f(1) / z32).astype(np.float64)
    delta = np.where(np.abs(z - z32) < 0.45 * 2.0 ** -23, 1 / z - s32, 0)      # z away from a tie of its rounding
    i = np.argmax(delta)
    assert delta[i] > 2.0 ** -24
    b0 = f(0.01 - s32[i])
    c0 = s32[i] + np.float64(b0)      # expert 0's choice in fp32, where the difference is exact; delta more in truth
    logits = torch.tensor([[0.0, low[i], -40.0, -40.0] + [-60.0] * 4])
    bias = torch.tensor([b0, -1.0, c0 + 0.6 * delta[i], c0 + 0.3 * delta[i], 0, 0, 0, 0], dtype=torch.float32)
    say("router later choice", low[i], bias.tolist())
    ids, _ = check(logits, 1, "softmax", bias)
    assert ids[0].tolist() == [0]


# T > 16 E or E <= 128, K <= 14 and at most 16 groups: 16 lanes a token, of 4, 8, 16 and 32 values
@pytest.mark.parametrize("T,E,K,groups", [
    (4200, 256, 8, (1, 1, 1)), (4117, 256, 14, (8, 4, 2)), (3500, 200, 5, (1, 1, 1)), (2500, 150, 3, (10, 4, 1)),
    (8200, 512, 8, (1, 1, 1)), (8200, 512, 8, (8, 4, 2)), (6200, 384, 8, (1, 1, 1)), (6203, 384, 14, (16, 5, 1)),
    (5000, 301, 6, (1, 1, 1)), (4400, 259, 11, (7, 3, 2)), (900, 64, 8, (1, 1, 1)), (901, 128, 8, (16, 6, 2))])
def test_many_tokens_in_16_lanes(T, E, K, groups):
    say("router 16 lanes", T, E, K, groups)
    kw = dict(zip(("n_group", "topk_group", "group_top"), groups))
    g = torch.Generator().manual_seed(T)
    logits, bias = 2 * torch.randn(T, E, generator=g), 0.1 * torch.randn(E, generator=g)
    logits[7, ::2] = -INF      # masked rows among them, and equal choices
    logits[8, 5:] = NAN
    logits[9] = 0
    logits[10, 3] = INF
    logits[11] = torch.finfo(torch.float32).min
    logits[12] = 1 + 2.0 ** -23 * torch.randperm(E, generator=g)
    logits[13] = -100
    half = logits.clamp(-1e30, 1e30).bfloat16()
    # the oracle goes token by token: the first and last rows and a thousand between them
    kw["rows"] = np.unique(np.r_[:40, T - 40:T, np.random.default_rng(T).integers(0, T, 1000)])
    check(logits, K, "softmax", **kw)
    check(logits, K, "sigmoid", bias, **kw)
    check(logits, K, "softmax", bias, renormalize=False, **kw)
    check(half, K, "softmax", renormalize=False, **kw)
    check(half, K, "sigmoid", bias, scale=2.5, **kw)
    check(half, K, "sigmoid", **kw)
