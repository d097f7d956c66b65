"""The 4-bit and mixture calls record nothing for autograd, and warn where it would want a gradient."""

import warnings

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import cuda, gen, weight

pytestmark = pytest.mark.gpu


def calls():
    w = bw.q4_upload(*(cuda(t) for t in weight(1, (4,), 128, 128, 64, True)))
    dense = bw.q4_upload(*(cuda(t) for t in weight(2, (), 64, 128, 64, True)))
    x = torch.randn((8, 128), generator=gen(3)).cuda()
    idx = torch.randint(0, 4, (8, 2), generator=gen(4)).int().cuda()
    wts, logits = torch.rand((8, 2), generator=gen(5)).cuda(), torch.randn((8, 4), generator=gen(6)).cuda()
    return [("x", x, lambda t: bw.q4_gemm(dense, t)), ("x", x, lambda t: bw.q4_moe(t, idx, wts, w, w, w)),
            ("weights", wts, lambda t: bw.q4_moe(x, idx, t, w, w, w)), ("logits", logits, lambda t: bw.moe_route(t, 2)[1])]


def test_a_lost_gradient_is_warned_of():
    note("[q4] inputs that require gradients")
    for name, t, call in calls():
        want = call(t)
        asks = t.clone().requires_grad_()
        with pytest.warns(UserWarning, match=f"no gradients?, but {name} require"):
            y = call(asks)
        assert torch.equal(y, want) and not y.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            call(t), call(asks.detach())
            with torch.no_grad():
                call(asks)
            with pytest.raises(UserWarning):
                call(asks)


def test_the_routers_gradient_takes_logits_that_require_one():
    logits = torch.randn((8, 4), generator=gen(7)).cuda().requires_grad_()
    note("[moe_route_backward] logits that require a gradient")
    with torch.no_grad():
        idx, w = bw.moe_route(logits, 2)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        logits.backward(bw.moe_route_backward(logits, idx, torch.ones_like(w)))
    want = torch.autograd.grad(torch.softmax(logits, 1).gather(1, idx.long()).sum(), logits)[0]
    # f32 on both sides: a few roundings of terms below 1
    assert float((logits.grad - want).abs().max()) <= 16 * 2.0 ** -24
