"""moe_router_topk on the GPU against the float64 oracle.

Chosen experts must be equal.  Weights: a score is held to (2 |x| + 16) * 2^-24 relative for logits (softmax: their
distance from the row's largest) of up to |x|: the argument of the exponential, rounded to fp32, carries |x| 2^-24
into it, and exponential, sum, quotient, renormalisation and scale add a few roundings each.
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


def check(logits, K, score, bias=None, **kw):
    ids, w = fm.moe_router_topk(logits.cuda(), K, SCORES[score], bias=None if bias is None else bias.cuda(), **kw)
    torch.cuda.synchronize()
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    rid, rw = router_reference(logits.double().numpy(), K, score, None if bias is None else bias.double().numpy(),
                               **kw)
    assert np.array_equal(ids, rid), f"rows {np.flatnonzero((ids != rid).any(1))[:8]}"
    x = logits.double().numpy()
    finite = np.where(np.isfinite(x), x, 0.0)
    reach = np.abs(finite).max(1) * (2 if score == "softmax" else 1)
    assert np.all(np.abs(w - rw) <= np.abs(rw) * ((2 * reach + 16) * 2.0 ** -24)[:, None] + 1e-38)
    return ids, w


def make(T, E, seed, dtype=torch.float32, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(T, E, generator=g)).to(dtype), 0.1 * torch.randn(E, generator=g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (5, 60, 4), (3, 64, 8), (33, 65, 6), (64, 128, 8), (65, 256, 8),
                                   (4, 257, 8), (7, 384, 10), (2, 1000, 16), (3, 1024, 64), (2, 64, 64), (1001, 40, 3)])
def test_shapes(T, E, K, score, dtype):
    say("router", T, E, K, score, dtype)
    logits, bias = make(T, E, T + E, dtype)
    check(logits, K, score)
    check(logits, K, score, bias)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,K", [
    (256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (64, 8, 3, 2, 6), (160, 8, 3, 1, 6), (60, 4, 1, 2, 15), (72, 3, 2, 2, 8),
    (1024, 64, 3, 2, 48), (32, 32, 5, 1, 5), (512, 2, 1, 2, 8), (16, 4, 4, 2, 16)])
def test_groups(E, n_group, topk_group, group_top, K, score, biased, dtype):
    say("router groups", E, n_group, topk_group, group_top, K, score, biased, dtype)
    logits, bias = make(75, E, E + K, dtype)
    check(logits, K, score, bias if biased else None, n_group=n_group, topk_group=topk_group, group_top=group_top,
          scale=2.5)


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("renormalize", [False, True])
def test_weights(score, renormalize):
    logits, bias = make(50, 96, 5)
    check(logits, 7, score, renormalize=renormalize, scale=1.0)
    check(logits, 7, score, bias, renormalize=renormalize, scale=-0.5)


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_ties_go_to_the_lowest_index(score, dtype):
    logits = torch.zeros(4, 200, dtype=dtype)
    logits[1] = torch.arange(200) % 3
    logits[2] = -(torch.arange(200) // 50).to(dtype)
    logits[3, 150:] = 1
    logits[0, ::3] = -0.0
    ids, _ = check(logits, 8, score)
    assert ids[0].tolist() == list(range(8))
    check(logits, 8, score, torch.zeros(200))
    check(logits, 8, score, n_group=4, topk_group=2, group_top=2)
    check(logits, 8, score, torch.zeros(200), n_group=4, topk_group=2, group_top=2)


@pytest.mark.parametrize("score", list(SCORES))
def test_close_scores(score):
    """Logits one fp32 step apart, saturated scores, and choices that differ far below fp32's step."""
    E = 256
    steps = torch.arange(E, dtype=torch.float32) * 2.0 ** -23
    one = (1 + steps[torch.randperm(E, generator=torch.Generator().manual_seed(1))]).view(1, E)
    far = 30 + one
    logits = torch.cat([one, far, -far, one * 2.0 ** -30, one * 1e30])
    check(logits, 8, score, renormalize=False)
    bias = torch.full((E,), 0.5)
    check(logits[:1], 8, score, bias)
    check(logits[:1], 8, score, bias, n_group=8, topk_group=4, group_top=2)
    check(logits[:1], 8, score, None, n_group=8, topk_group=4, group_top=2)
    # the bias and the score nearly cancel: the order hangs on the scores' last bits
    g = torch.Generator().manual_seed(2)
    x = torch.randn(64, E, generator=g)
    s = torch.softmax(x[:1].double(), 1) if score == "softmax" else torch.sigmoid(x[:1].double())
    check(x[:1], 8, score, (1.0 - s[0]).float())
    check(x, 8, score, (1.0 - s[0]).float())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,n_group,K", [(160, 8, 8), (66, 6, 5), (231, 7, 9), (500, 10, 14), (384, 12, 8), (51, 17, 4),
                                         (48, 16, 3), (63, 63, 20), (1023, 33, 8), (4, 2, 2), (392, 8, 7),
                                         (240, 6, 8), (252, 12, 8), (60, 5, 6), (120, 3, 8), (448, 14, 8), (990, 6, 30)])
def test_groups_of_any_size(E, n_group, K, biased, dtype):
    """Groups that are no whole numbers of lanes, or vectors, or fewer than lanes; rows that start unaligned."""
    say("router group sizes", E, n_group, K, biased, dtype)
    logits, bias = make(70, E, 3 * E + K, dtype)
    for score in SCORES:
        for group_top in range(1, min(2, E // n_group) + 1):
            kw = dict(n_group=n_group, topk_group=max(1, n_group // 2), group_top=group_top)
            check(logits, K, score, bias if biased else None, **kw)
    far = torch.empty(70 * E + 1, dtype=dtype, device="cuda")[1:].view(70, E)
    far.copy_(logits)
    ids, w = fm.moe_router_topk(far, K, fm.SCORE_SIGMOID, bias=bias.cuda() if biased else None)
    ids2, w2 = fm.moe_router_topk(logits.cuda(), K, fm.SCORE_SIGMOID, bias=bias.cuda() if biased else None)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("E,n_group,topk_group", [(256, 8, 4), (128, 16, 5), (512, 4, 1)])
def test_close_groups(E, n_group, topk_group, group_top, score):
    """Groups of the same logits in another order, moved by a few of fp32's smallest steps; equal groups; biases that
    are far larger than the sums of a group's best choices."""
    say("router close groups", E, n_group, topk_group, group_top, score)
    g = torch.Generator().manual_seed(E + group_top)
    G = E // n_group
    one = torch.randn(40, 1, G, generator=g).expand(40, n_group, G)
    order = torch.argsort(torch.rand(40, n_group, G, generator=g), 2)
    logits = torch.gather(one, 2, order)
    logits[20:] *= 1 + 2.0 ** -22 * torch.randint(-2, 3, (20, n_group, 1), generator=g)
    logits = logits.reshape(40, E).contiguous()
    kw = dict(n_group=n_group, topk_group=topk_group, group_top=group_top)
    check(logits, 8, score, **kw)
    check(logits, 8, score, torch.zeros(E), **kw)
    check(logits, 8, score, torch.full((E,), 0.3), **kw)
    check(logits, 8, score, torch.full((E,), -1000.0), **kw)
    check(logits.bfloat16(), 8, score, torch.full((E,), 0.3), **kw)
    # +1000 and -1000 on a group's best two: their sums are about a score's size
    bias = torch.full((n_group, G), -2000.0)
    bias[:, 1], bias[:, G - 1] = 1000.0, -1000.0
    check(torch.randn(400, E, generator=g), 8, score, bias.view(-1), **kw)
    bias[:, 1] += 2.0 ** -14 * torch.arange(n_group) % 3
    check(0.001 * torch.randn(400, E, generator=g), 8, score, bias.view(-1), **kw)


@pytest.mark.parametrize("score", list(SCORES))
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("groups", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_masked_logits(score, biased, groups):
    """-inf, NaN, +inf and the type's lowest value; rows with fewer experts than slots, and with none."""
    say("router masks", score, biased, groups)
    n_group, topk_group, group_top = groups
    logits, bias = make(12, 64, 21)
    logits[0] = -INF
    logits[1] = NAN
    logits[2, 3:] = -INF
    logits[3, ::2] = -INF
    logits[4, 5] = INF
    logits[5, 5], logits[5, 40] = INF, INF
    logits[6, 5] = NAN
    logits[7] = torch.finfo(torch.float32).min
    logits[8, 8:] = torch.finfo(torch.float32).min
    logits[9, 1:] = -INF
    logits[10, :16] = -INF
    kw = dict(n_group=n_group, topk_group=topk_group, group_top=group_top)
    ids, w = check(logits, 8, score, bias if biased else None, **kw)
    assert (ids[0] == -1).all() and (w[0] == 0).all() and (ids[1] == -1).all()
    if biased:
        bias[7], bias[9], bias[11] = -INF, NAN, INF
        check(logits, 8, score, bias, **kw)


def test_softmax_of_far_logits_underflows_to_zero():
    logits = torch.full((1, 16), -1e4)
    logits[0, 3] = 1e4
    ids, w = check(logits, 4, "softmax")
    assert ids[0].tolist() == [3, 0, 1, 2] and w[0].tolist() == [1, 0, 0, 0]
    logits = torch.full((1, 16), -2000.0)     # sigmoid: every score is 0, and so is their sum
    ids, w = check(logits, 4, "sigmoid")
    assert ids[0].tolist() == [0, 1, 2, 3] and w[0].tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("T,E,K,groups", [(5000, 256, 8, (8, 4, 2)), (5000, 256, 8, (8, 3, 1)), (5003, 128, 6, (1, 1, 1)),
                                          (3001, 64, 7, (4, 2, 2)), (2000, 512, 15, (8, 4, 2)),
                                          (1501, 192, 15, (6, 2, 2)), (1200, 1000, 20, (1, 1, 1))])
def test_many_tokens(T, E, K, groups):
    """Enough rows that close scores occur among them."""
    say("router many", T, E, K, groups)
    kw = dict(zip(("n_group", "topk_group", "group_top"), groups))
    logits, bias = make(T, E, 77)
    check(logits, K, "sigmoid", bias, **kw)
    check(logits, K, "softmax", bias, **kw)
    check(logits, K, "softmax", **kw)
    check(logits.bfloat16(), K, "softmax", renormalize=False, **kw)
    check(logits.bfloat16(), K, "sigmoid", bias, **kw)
    check(logits * 2.0 ** -12, K, "sigmoid", **kw)
    check(logits * 2.0 ** -12, K, "sigmoid", bias * 2.0 ** -12, **kw)


def test_unaligned_views():
    """Rows that no 16-byte vector can read."""
    flat = make(40, 256, 3)[0].reshape(-1)
    for off in (1, 2, 3):
        logits = flat[off:off + 39 * 256].view(39, 256)
        dev = flat.cuda()[off:off + 39 * 256].view(39, 256)
        ids, w = fm.moe_router_topk(dev, 8)
        rid, _ = router_reference(logits.double().numpy(), 8, "softmax")
        assert np.array_equal(ids.cpu().numpy(), rid)


def test_given_outputs_stream_and_graph():
    logits, bias = (t.cuda() for t in make(300, 256, 8))
    kw = dict(bias=bias, n_group=8, topk_group=4, group_top=2)
    want = fm.moe_router_topk(logits, 8, fm.SCORE_SIGMOID, **kw)
    ids, w = torch.empty_like(want[0]), torch.empty_like(want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fm.moe_router_topk(logits, 8, fm.SCORE_SIGMOID, ids=ids, weights=w, **kw)
    s.synchronize()
    assert torch.equal(ids, want[0]) and torch.equal(w, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fm.moe_router_topk(logits, 8, fm.SCORE_SIGMOID, **kw)
    for seed in (1, 2, 3):
        logits.copy_(make(300, 256, seed)[0])
        g.replay()
        torch.cuda.synchronize()
        want = fm.moe_router_topk(logits, 8, fm.SCORE_SIGMOID, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals():
    logits, bias = (t.cuda() for t in make(4, 64, 8))
    f = fm.moe_router_topk
    with pytest.raises(TypeError):
        f(logits.half(), 4)
    with pytest.raises(TypeError):
        f(logits, 4, bias=bias.bfloat16())
    with pytest.raises(ValueError):
        f(logits, 4, bias=bias[:63].contiguous())
    with pytest.raises(ValueError):
        f(logits.t(), 4)
    with pytest.raises(ValueError):
        f(logits, 4, bias=bias.cpu())
    with pytest.raises(ValueError):
        f(logits, 4, ids=torch.empty(4, 5, dtype=torch.int32, device="cuda"))
    for kw in (dict(K=0), dict(K=65), dict(K=17, n_group=4, topk_group=1), dict(K=4, n_group=3),
               dict(K=4, n_group=4, topk_group=5), dict(K=4, n_group=4, topk_group=0), dict(K=4, group_top=3),
               dict(K=1, n_group=64, topk_group=2, group_top=2), dict(K=4, score=2), dict(K=4, scale=INF)):
        with pytest.raises(fm.Fp8MoeError):
            f(logits, **kw)
    ids, w = f(logits[:0], 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
