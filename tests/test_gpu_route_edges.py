"""The router and its gradient where f32 scores decide wrongly, saturate, underflow or are not finite.

Indices are whole numbers, compared with the definition in f64.  Gradients are compared element by element in
relative terms.  Renormalised, w_j = c_j / sum c by exponents relative to the largest chosen logit: an argument is off by half
a step of the chosen logits' span S (S 2^-24), exp, sum, quotient and the factor 1 - p by at most 12 steps of 2^-24 more, for
w_j and again for each w_i of the sum; so (2 S + 32) 2^-24 of w_j (|dw_j| + sum w_i |dw_i|).  Sigmoid without
renormalising: dw p (1 - p), each factor a few steps: 16 2^-24 of the value.  Results below the normal range: 2^-126 2^-22.
"""

import math

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import cuda, gen, route64

pytestmark = pytest.mark.gpu
INF, NAN = math.inf, math.nan


def check(logits, k, what, bias=None, score="sigmoid", groups=1, keep=1, group_top=1):
    note(f"[moe_route] {what}")
    idx, w = bw.moe_route(logits.cuda(), k, bias=cuda(bias), score=score, groups=groups, keep=keep, group_top=group_top)
    want, want_w = route64(logits, k, bias, score, groups, keep, group_top, False)
    assert torch.equal(idx.cpu(), want), what
    fin = logits[torch.isfinite(logits)].double()
    # as test_gpu_moe's: (L + 12) 2^-23 of the weight
    tol = (float(fin.abs().max()) + 12) * 2.0 ** -23 * want_w + 2.0 ** -149
    assert ((w.cpu().double() - want_w).abs() <= tol).all(), what


def test_sigmoid_scores_below_f32s_normal_range():
    """Sums of scores near 2^-126: e^-87 + e^-300 against twice e^-87.5."""
    check(torch.tensor([[-87.0, -300.0, -87.5, -87.5]]), 2, "sums near 2^-126", groups=2, keep=1, group_top=2)
    logits = -85 - 25 * torch.rand((300, 64), generator=gen(1))
    check(logits, 6, "all scores small", groups=8, keep=3, group_top=2)
    bias = torch.randint(0, 4, (64,), generator=gen(2)) * 2.0 ** -127
    check(logits, 6, "small biases too", bias, groups=8, keep=3, group_top=2)
    check(logits, 6, "without groups", bias)


def test_softmax_scores_below_f32s_normal_range():
    logits = -85 - 25 * torch.rand((300, 64), generator=gen(3))
    logits[:, 5] = 0
    bias = torch.zeros(64)
    bias[5] = -INF
    check(logits, 6, "softmax, all but one small", bias, "softmax")
    check(logits, 6, "softmax groups", bias, "softmax", groups=8, keep=3, group_top=2)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_saturated_scores_tie_as_in_the_definition(score):
    """Two best keys to a group: the keys are scores, and sigmoid(40) = sigmoid(50) = 1 in f64."""
    check(torch.tensor([[40.0, 50.0, 0.0, 0.0]]), 2, f"saturated {score}", None, score, 2, 1, 2)
    logits = torch.randint(20, 60, (300, 64), generator=gen(4)).float()
    check(logits, 8, f"saturated rows {score}", None, score, 8, 3, 2)
    logits = torch.randint(0, 3, (300, 64), generator=gen(5)) * 1e-20
    check(logits, 8, f"scores that agree {score}", None, score, 8, 3, 2)


def test_long_sums_of_a_softmax_do_not_decide():
    """33 groups of 31: each lane adds 30 terms that f32 loses, 1.8e-6 of the sum, and a bias puts two keys within that."""
    groups, n = 33, 31
    logits = torch.full((1, groups, n), -16.65)
    logits[:, :, 0] = 0
    p = float(torch.softmax(logits.double().flatten(), 0)[0])
    bias = torch.full((groups, n), -INF)
    bias[0, 0] = -1 / 33
    true_key = p + float(bias[0, 0])
    other = float(torch.softmax(logits.double().flatten(), 0)[n + 1])
    bias[1, 1] = true_key + 1.2e-8 - other
    check(logits.view(1, -1), 2, "long sums", bias.flatten(), "softmax", groups, groups, 1)
    check(logits.view(1, -1), 2, "long sums, one group", bias.flatten(), "softmax")


@pytest.mark.parametrize("groups,keep,group_top,bias", [(1, 1, 1, True), (4, 2, 2, False), (4, 2, 1, True)])
def test_softmax_of_rows_that_are_not_finite(groups, keep, group_top, bias):
    """A NaN logit, and one of +inf, make every score NaN: all weights show it, whatever the keys are."""
    logits = torch.randn((4, 32), generator=gen(6))
    logits[1, 9], logits[2, 20] = NAN, INF
    b = 0.1 * torch.randn(32, generator=gen(7)) if bias else None
    note(f"[moe_route] rows that are not finite groups={groups} top={group_top} bias={bias}")
    for renorm in (False, True):
        idx, w = (v.cpu() for v in bw.moe_route(logits.cuda(), 4, bias=cuda(b), groups=groups, keep=keep,
                                                group_top=group_top, renorm=renorm))
        assert w[[1, 2]].isnan().all() and torch.isfinite(w[[0, 3]]).all()
        assert ((idx >= 0) & (idx < 32)).all()


def gradient64(logits, idx, dw, score, renorm):
    """dlogits from the closed forms in f64, with 1 - p formed without cancelling; and the terms' magnitudes."""
    l, dw = logits.double(), dw.double()
    on = (idx >= 0) & (idx < l.shape[1])
    at = idx.long().clamp(0, l.shape[1] - 1)
    c = torch.where(on, l.gather(1, at), -INF)
    p = torch.sigmoid(c) if score == "sigmoid" else None
    q = torch.sigmoid(-c) if score == "sigmoid" else torch.ones_like(c)
    if renorm:
        most = c.max(1, keepdim=True).values
        w = torch.exp(c - most) * (q / torch.sigmoid(-most) if score == "sigmoid" else 1)  # p_j over the largest p
        w = torch.where(on, w, 0.0)
        w = w / w.sum(1, keepdim=True)
        dw = torch.where(on, dw, 0.0)
        mean, size = (w * dw).sum(1, keepdim=True), (w * dw.abs()).sum(1, keepdim=True)
        v, mag = w * (dw - mean) * q, w * (dw.abs() + size) * q
    else:
        v = torch.where(on, dw * p * q, 0.0)
        mag = v.abs()
    out = torch.zeros_like(l).scatter_add(1, at, torch.where(on, v, 0.0))
    return out, torch.zeros_like(l).scatter_add(1, at, torch.where(on, mag, 0.0))


def check_gradient(logits, idx, dw, score, renorm, what):
    note(f"[moe_route_backward] {what} {score} renorm={renorm}")
    got = bw.moe_route_backward(logits.cuda(), idx.cuda(), dw.cuda(), score=score, renorm=renorm).cpu().double()
    want, mag = gradient64(logits, idx, dw, score, renorm)
    c = logits.double().gather(1, idx.long())
    span = (c.max(1).values - c.min(1).values)[:, None]
    tol = ((2 * span + 32) if renorm else 16) * 2.0 ** -24 * mag + 2.0 ** -148
    assert torch.isfinite(got).all(), what
    assert ((got - want).abs() <= tol).all(), (what, float(((got - want).abs() / tol).max()))


@pytest.mark.parametrize("below", [0, 60, 88, 95, 103, 300, 600])
def test_renormalised_softmax_gradient_far_below_the_maximum(below):
    """Chosen experts whose scores are small beside the row's largest, which a bias or a dropped group keeps out."""
    t, e, k = 20, 40, 5
    logits = torch.randn((t, e), generator=gen(8))
    idx = torch.stack([torch.randperm(e - 1, generator=gen(20 + i))[:k] for i in range(t)]).int()
    logits[:, e - 1] = below
    dw = torch.randn((t, k), generator=gen(9))
    check_gradient(logits, idx, dw, "softmax", True, f"{below} below")


@pytest.mark.parametrize("at", [-600, -300, -100, -88, -60, -20, 0, 20, 60, 300])
def test_renormalised_sigmoid_gradient_of_large_logits(at):
    t, e, k = 20, 40, 5
    logits = torch.randn((t, e), generator=gen(10)) + at
    idx = torch.topk(logits, k, dim=1).indices.int()
    check_gradient(logits, idx, torch.randn((t, k), generator=gen(11)), "sigmoid", True, f"logits near {at}")


def test_renormalised_sigmoid_gradient_of_mixed_signs():
    t, e, k = 50, 64, 6
    logits = 30 * torch.randn((t, e), generator=gen(12))
    idx = torch.topk(logits, k, dim=1).indices.int()
    check_gradient(logits, idx, torch.randn((t, k), generator=gen(13)), "sigmoid", True, "mixed signs")


@pytest.mark.parametrize("at", [-60, -20, 0, 5, 10, 16, 20, 60])
def test_sigmoid_gradient_of_large_logits(at):
    t, e, k = 20, 40, 5
    logits = torch.randn((t, e), generator=gen(14)) + at
    idx = torch.topk(logits, k, dim=1).indices.int()
    check_gradient(logits, idx, torch.randn((t, k), generator=gen(15)), "sigmoid", False, f"logits near {at}")


def test_renormalised_gradient_of_rows_that_leave_nothing():
    """Chosen logits of -inf have no weight: their rows' gradients are 0, and other slots' as if they were dropped."""
    logits = torch.randn((3, 16), generator=gen(16))
    logits[0] = -INF
    logits[1, :4] = -INF
    idx = torch.tensor([[0, 1, 2], [0, 5, 6], [7, 8, 9]], dtype=torch.int32)
    dw = torch.randn((3, 3), generator=gen(17))
    note("[moe_route_backward] rows that leave nothing")
    for score in ("softmax", "sigmoid"):
        got = bw.moe_route_backward(logits.cuda(), idx.cuda(), dw.cuda(), score=score, renorm=True).cpu()
        assert (got[0] == 0).all() and (got[1, :4] == 0).all() and torch.isfinite(got).all()
        dropped = idx.clone()
        dropped[1, 0] = -1
        want, mag = gradient64(logits, dropped, dw, score, True)
        assert ((got[1:].double() - want[1:]).abs() <= 64 * 2.0 ** -24 * mag[1:]).all()
