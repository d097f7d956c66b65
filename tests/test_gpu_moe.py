"""GPU parity of the router, its gradient and the experts' products with 64-bit references.

Tolerances.  Chosen experts are compared as whole numbers.  Weights whose keys are sums of
scores come from f64 and are rounded once (2^-24); the others from f32: the argument of
exp is off by up to half a step of its size (L = the largest distance to the maximum,
or |l| for a sigmoid), exp, sum and quotient by a few more steps: (L + 12) 2^-23 of the
weight.  The gradient likewise, (L + 16) 2^-23 of the sum of the magnitudes of its terms, plus the
rounding to its type.  The experts' products: f32 sums in all three products,
2^-18 of the result's norm for f32; for 16-bit types eps/2 for the result and
eps(f16) for silu(g) u where it is held in f16, with, for bfloat16, weights rounded to
f16 on the way (2^-11 for each of three products).
"""

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import DTYPES, cuda, dequant64, gen, moe64, route64, route_weights64, weight

pytestmark = pytest.mark.gpu
INF = float("inf")


def check_route(logits, k, what, bias=None, score="softmax", groups=1, keep=1, group_top=1, renorm=False):
    t, e = logits.shape
    idx = torch.full((t * k + 8,), -77, dtype=torch.int32, device="cuda")
    wts = torch.full((t * k + 8,), float("nan"), device="cuda")
    gi, gw = bw.moe_route(logits.cuda(), k, bias=cuda(bias), score=score, groups=groups, keep=keep, group_top=group_top,
                          renorm=renorm, idx=idx[: t * k].view(t, k), weights=wts[: t * k].view(t, k))
    torch.cuda.synchronize()
    assert (idx[t * k:] == -77).all() and torch.isnan(wts[t * k:]).all(), "write past the end"
    want_i, want_w = route64(logits, k, bias, score, groups, keep, group_top, renorm)
    gi, gw = gi.cpu(), gw.cpu()
    assert torch.equal(gi, want_i), what
    fin = logits[torch.isfinite(logits)].double()
    span = float((fin.max() - fin.min()).clamp(min=fin.abs().max())) if fin.numel() else 0.0
    tol = (span + 12) * 2.0 ** -23 * want_w.abs() + 2.0 ** -149
    same = (gw.double() - want_w).abs() <= tol
    assert (same | (gw.isnan() & want_w.isnan())).all(), what
    return gi, gw


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,e,k,groups,keep,group_top,bias,renorm",
                         [(1, 1, 1, 1, 1, 1, False, False), (7, 8, 8, 1, 1, 1, False, True),
                          (65, 60, 6, 1, 1, 1, True, False), (33, 64, 4, 4, 2, 1, False, True),
                          (130, 256, 8, 8, 4, 2, True, True), (50, 160, 6, 8, 3, 2, False, False),
                          (9, 129, 5, 3, 2, 2, True, True), (5, 1000, 64, 4, 4, 1, True, False),
                          (40, 77, 7, 7, 5, 1, True, True), (3, 1024, 10, 64, 20, 2, True, True)])
def test_route(t, e, k, groups, keep, group_top, bias, renorm, score, dtype):
    logits = torch.randn((t, e), generator=gen(1)).to(DTYPES[dtype])
    b = 0.1 * torch.randn(e, generator=gen(2)) if bias else None
    note(f"[moe_route] T={t} E={e} k={k} {score} groups={groups} keep={keep} top={group_top} bias={bias} {dtype}")
    check_route(logits, k, f"T={t} E={e}", b, score, groups, keep, group_top, renorm)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,keep,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_equal_keys_take_the_lower_index(score, groups, keep, group_top):
    logits = torch.randint(-2, 3, (200, 64), generator=gen(3)).float()
    logits[0] = 0
    note(f"[moe_route] ties {score} groups={groups}")
    check_route(logits, 8, "ties", None, score, groups, keep, group_top, True)
    check_route(logits, 8, "ties with an equal bias", torch.zeros(64), score, groups, keep, group_top, True)


def test_route_near_ties_are_decided_in_f64():
    """Sums of a score and a bias that agree in f32 and differ in f64."""
    e = 128
    logits = torch.zeros((64, e))
    logits += torch.arange(64)[:, None] * 1e-3
    bias = torch.full((e,), 2.0 ** -30)
    bias[5] = 2.0 ** -28
    bias[100] = 2.0 ** -27
    note("[moe_route] near ties")
    gi, _ = check_route(logits, 3, "near ties", bias, "sigmoid")
    assert (gi == torch.tensor([100, 5, 0], dtype=torch.int32)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,keep,group_top", [(1, 1, 1), (4, 2, 2)])
def test_route_masked_experts(score, bias, groups, keep, group_top):
    """Logits of -inf: rows that leave fewer experts than slots, one, and none; the type's lowest value is no mask."""
    logits = torch.randn((12, 32), generator=gen(4))
    logits[0] = -INF
    logits[1, 1:] = -INF
    logits[2, :29] = -INF
    logits[3, 8:16] = -INF
    logits[4] = torch.finfo(torch.float32).min
    logits[5, :31] = torch.finfo(torch.float32).min
    logits[6, 9] = INF if score == "sigmoid" else 80.0
    b = 0.1 * torch.randn(32, generator=gen(5)) if bias else None
    note(f"[moe_route] masks {score} bias={bias} groups={groups}")
    gi, gw = check_route(logits[:4], 4, "masks", b, score, groups, keep, group_top, True)
    assert (gi[0] == -1).all() and (gw[0] == 0).all()
    assert (gi[1, 1:] == -1).all() and (gw[1, 1:] == 0).all()
    got_i, got_w = bw.moe_route(logits[4:].cuda(), 4, bias=cuda(b), score=score, groups=groups, keep=keep,
                                group_top=group_top, renorm=False)
    want_i, want_w = route64(logits[4:], 4, b, score, groups, keep, group_top, False)
    assert torch.equal(got_i.cpu(), want_i)
    assert torch.allclose(got_w.cpu().double(), want_w, rtol=2.0 ** -15, atol=2.0 ** -140)


def test_route_nan_shows():
    logits = torch.randn((4, 64), generator=gen(6))
    logits[1, 7] = float("nan")
    note("[moe_route] NaN logits")
    for score in ("softmax", "sigmoid"):
        gi, gw = (v.cpu() for v in bw.moe_route(logits.cuda(), 4, score=score))
        assert gi[1, 0] == 7 and torch.isnan(gw[1, 0])
        assert torch.isfinite(gw[[0, 2, 3]]).all() and (gi >= 0).all() and (gi < 64).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_many_tokens(score, dtype):
    """Every index of a long prompt, against torch's stable sort in f64."""
    t, e, k = 8192, 256, 8
    logits = torch.randn((t, e), generator=gen(7)).to(DTYPES[dtype]).cuda()
    bias = (0.1 * torch.randn(e, generator=gen(8))).cuda()
    note(f"[moe_route] T={t} {score} {dtype}")
    l = logits.double()
    p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    key = p + bias.double()
    by = key.view(t, 8, 32)
    best = by.topk(2, 2).values.sum(2)
    kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :4]
    allowed = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
    key = torch.where(allowed[:, :, None], by, -INF).view(t, e)
    want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    idx, w = bw.moe_route(logits, k, bias=bias, score=score, groups=8, keep=4, group_top=2, renorm=True)
    assert torch.equal(idx.long(), want)
    c = p.gather(1, want)
    assert torch.allclose(w.double(), c / c.sum(1, keepdim=True), rtol=2.0 ** -23, atol=0)


def check_backward(logits, idx, dw, score, renorm, dtype, what):
    l64 = logits.double().requires_grad_()
    out = route_weights64(l64, idx, score, renorm)
    (want,) = torch.autograd.grad((out * dw.double()).sum(), l64)
    t, e = logits.shape
    base = torch.full((t * e + 8,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    got = bw.moe_route_backward(logits.cuda(), idx.cuda(), dw.cuda(), score=score, renorm=renorm,
                                dlogits=base[: t * e].view(t, e))
    torch.cuda.synchronize()
    assert torch.isnan(base[t * e:]).all(), "write past the end"
    got = got.cpu().double()
    # magnitudes of the terms: |dw| c / total twice (numerator and quotient), times p
    p = torch.softmax(l64.detach(), 1) if score == "softmax" else torch.sigmoid(l64.detach())
    on = (idx >= 0) & (idx < e)
    c = torch.where(on, p.gather(1, idx.long().clamp(0, e - 1)), 0.0)
    total = c.sum(1, keepdim=True) if renorm else torch.ones((t, 1), dtype=torch.float64)
    dc = torch.where(on, (dw.double().abs() + ((dw.double().abs() * c).sum(1, keepdim=True) / total if renorm else 0)), 0.0) / total
    mag = torch.zeros_like(p).scatter_add(1, idx.long().clamp(0, e - 1), dc)
    mag = p * (mag + (dc * c).sum(1, keepdim=True)) if score == "softmax" else mag * p
    span = float((logits.double().max() - logits.double().min()).abs())
    tol = (span + 16) * 2.0 ** -23 * mag + torch.finfo(DTYPES[dtype]).eps / 2 * want.abs() + 2.0 ** -25
    if dtype == "f32":
        tol = tol - 2.0 ** -25 + 1e-40
    assert ((got - want).abs() <= tol).all(), what
    return got, want


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (9, 8, 3), (130, 128, 8), (33, 250, 6), (5, 1024, 64), (1000, 64, 6)])
def test_route_backward(t, e, k, renorm, score, dtype):
    logits = torch.randn((t, e), generator=gen(9)).to(DTYPES[dtype])
    idx = torch.topk(logits.float(), k, dim=1).indices.int()
    dw = torch.randn((t, k), generator=gen(10))
    note(f"[moe_route_backward] T={t} E={e} k={k} {score} renorm={renorm} {dtype}")
    check_backward(logits, idx, dw, score, renorm, dtype, f"T={t} E={e}")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward_against_differences(score):
    """The kernel's gradient against central differences of the f64 forward (step 1e-5: error below 1e-9)."""
    t, e, k = 3, 12, 4
    logits = torch.randn((t, e), generator=gen(11))
    idx, _ = route64(logits, k, None, score, 1, 1, 1, True)
    dw = torch.randn((t, k), generator=gen(12))
    note(f"[moe_route_backward] differences {score}")
    got = bw.moe_route_backward(logits.cuda(), idx.cuda(), dw.cuda(), score=score, renorm=True).cpu().double()
    f = lambda l: (route_weights64(l, idx, score, True) * dw.double()).sum()  # noqa: E731
    for r in range(t):
        for i in range(e):
            d = torch.zeros((t, e), dtype=torch.float64)
            d[r, i] = 1e-5
            diff = (f(logits.double() + d) - f(logits.double() - d)) / 2e-5
            assert abs(float(diff - got[r, i])) <= 1e-9 + 32 * 2.0 ** -23 * float(dw[r].abs().sum())


def test_route_backward_dropped_and_repeated_slots():
    t, e, k = 6, 40, 4
    logits = torch.randn((t, e), generator=gen(13))
    idx = torch.topk(logits, k, dim=1).indices.int()
    idx[0, 1] = -1
    idx[1] = -1
    idx[2, 2] = e  # past the last expert: no slot
    idx[3, 3] = idx[3, 0]
    dw = torch.randn((t, k), generator=gen(14))
    note("[moe_route_backward] dropped and repeated slots")
    for score in ("softmax", "sigmoid"):
        got, _ = check_backward(logits, idx, dw, score, False, "f32", score)
        assert (got[1] == 0).all()
        z = bw.moe_route_backward(logits.cuda(), idx.cuda(), dw.cuda(), score=score, renorm=True).cpu()
        assert (z[1] == 0).all() and torch.isfinite(z).all()


def test_route_and_backward_in_a_graph():
    t, e, k = 300, 64, 6
    logits = torch.randn((t, e), generator=gen(15)).cuda()
    dw = torch.randn((t, k), generator=gen(16)).cuda()
    idx = torch.empty((t, k), dtype=torch.int32, device="cuda")
    w, dl = torch.empty((t, k), device="cuda"), torch.empty((t, e), device="cuda")

    def work():
        bw.moe_route(logits, k, renorm=True, idx=idx, weights=w)
        bw.moe_route_backward(logits, idx, dw, renorm=True, dlogits=dl)

    note("[moe_route] graph")
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for rep in range(3):
        logits.copy_(torch.randn((t, e), generator=gen(17 + rep)))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (idx, w, dl)]
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (idx, w, dl))), rep


def experts(seed, e, d, f, group, zeros, dgroup=None):
    return (weight(seed, (e,), f, d, group, zeros), weight(seed + 1, (e,), f, d, group, zeros),
            weight(seed + 2, (e,), d, f, dgroup or group, zeros))


def check_moe(t, e, k, d, f, group, zeros, dtype, what, idx=None, dgroup=None, seed=20):
    gate, up, down = experts(seed, e, d, f, group, zeros, dgroup)
    x = torch.randn((t, d), generator=gen(seed + 3)).to(DTYPES[dtype])
    if idx is None:
        idx = torch.stack([torch.randperm(e, generator=gen(seed + 100 + i))[:k] for i in range(t)]).int()
        idx = torch.where(torch.rand((t, k), generator=gen(seed + 4)) < 0.1, -1, idx)
    idx = idx.int().contiguous()
    wts = torch.rand((t, k), generator=gen(seed + 5)) + 0.1
    handles = [bw.q4_upload(*(cuda(v) for v in w)) for w in (gate, up, down)]
    base = torch.full((t * d + 64,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    note(f"[q4_moe {what}] T={t} E={e} k={k} d={d} f={f} G={group} zeros={zeros} {dtype}")
    y = bw.q4_moe(x.cuda(), idx.cuda(), wts.cuda(), *handles, base[: t * d].view(t, d))
    torch.cuda.synchronize()
    assert torch.isnan(base[t * d:]).all(), "write past the end"
    want = moe64(x, idx, wts, *(dequant64(*w) for w in (gate, up, down)))
    y64 = y.cpu().double()
    gone = ~((idx >= 0) & (idx < e)).any(1)
    assert (y64[gone] == 0).all(), "tokens without slots"
    eps = torch.finfo(DTYPES[dtype]).eps
    tol = 2.0 ** -18 if dtype == "f32" else eps / 2 + 2.0 ** -10 + (3 * 2.0 ** -11 if dtype == "bf16" else 0)
    err = float((y64 - want).norm() / want.norm()) if want.norm() else float(y64.norm())
    note(f"  rel {err:.3g} (allowed {tol:.3g})")
    assert err <= tol, what
    rows = want.norm(dim=1) > 0
    if rows.any():  # no single token may be far off either
        worst = float(((y64 - want).norm(dim=1)[rows] / want.norm(dim=1)[rows]).max())
        assert worst <= 4 * tol, what
    again = bw.q4_moe(x.cuda(), idx.cuda(), wts.cuda(), *handles)
    assert torch.equal(y, again), "not deterministic"


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,e,k,d,f,group,zeros",
                         [(1, 4, 1, 128, 128, 128, False), (1, 16, 8, 256, 320, 64, True), (2, 8, 3, 288, 96, 32, True),
                          (4, 64, 8, 256, 128, 128, False), (33, 32, 4, 256, 192, 64, True), (5, 5, 5, 384, 256, 128, True),
                          (100, 4, 2, 256, 256, 32, False), (150, 8, 4, 320, 160, 32, True), (600, 4, 3, 256, 128, 128, False)])
def test_moe(t, e, k, d, f, group, zeros, dtype):
    check_moe(t, e, k, d, f, group, zeros, dtype, "sizes")


@pytest.mark.parametrize("t", [1, 6, 300])
def test_moe_dropped_slots_and_experts_out_of_range(t):
    e, k = 6, 3
    idx = torch.randint(-2, e + 2, (t, k), generator=gen(30))
    idx[0] = -1
    check_moe(t, e, k, 128, 128, 64, False, "bf16", "dropped", idx=idx)


@pytest.mark.parametrize("t,k", [(1, 4), (3, 2), (200, 2)])
def test_moe_one_expert_takes_all(t, k):
    """Every slot on one expert (a token may name it several times): its rows fill many tiles, the others none."""
    idx = torch.full((t, k), 2)
    check_moe(t, 5, k, 128, 96, 32, True, "bf16", "one expert", idx=idx)


def test_moe_down_with_other_groups():
    check_moe(40, 6, 2, 256, 192, 128, True, "f16", "other groups", dgroup=32)


@pytest.mark.parametrize("t", [1, 50, 500])
def test_moe_large_activations(t):
    """silu(g) u far beyond f16's range, in bfloat16, where the result is in range again."""
    e, k, d, f = 4, 2, 128, 128
    gate, up, down = experts(40, e, d, f, 64, False)
    up = (up[0], (up[1].float() * 300).half(), None)
    down = (down[0], (down[1].float() / 300).half(), None)
    x = (torch.randn((t, d), generator=gen(41)) * 300).bfloat16()
    idx = torch.stack([torch.randperm(e, generator=gen(50 + i))[:k] for i in range(t)]).int()
    wts = torch.rand((t, k), generator=gen(42)) + 0.1
    note(f"[q4_moe] large activations T={t}")
    y = bw.q4_moe(x.cuda(), idx.cuda(), wts.cuda(), *[bw.q4_upload(*(cuda(v) for v in w)) for w in (gate, up, down)])
    want = moe64(x, idx, wts, *(dequant64(*w) for w in (gate, up, down)))
    err = float((y.cpu().double() - want).norm() / want.norm())
    assert err <= 2.0 ** -8 + 2.0 ** -10 + 3 * 2.0 ** -11, err


@pytest.mark.parametrize("t", [1, 20, 400])
def test_moe_in_a_graph_and_on_another_stream(t):
    e, k, d, f = 8, 2, 256, 128
    handles = [bw.q4_upload(*(cuda(v) for v in w)) for w in experts(60, e, d, f, 64, True)]
    x = torch.randn((t, d), generator=gen(61)).bfloat16().cuda()
    idx = torch.randint(0, e, (t, k), generator=gen(62)).int().cuda()
    wts = torch.rand((t, k), generator=gen(63)).cuda()
    y = torch.empty_like(x)
    note(f"[q4_moe] graph T={t}")
    bw.q4_moe(x, idx, wts, *handles, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bw.q4_moe(x, idx, wts, *handles, y)
    for rep in range(4):
        x.copy_(torch.randn((t, d), generator=gen(64 + rep)).bfloat16())
        idx.copy_(torch.randint(-1, e, (t, k), generator=gen(70 + rep)).int())
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bw.q4_moe(x, idx, wts, *handles)), rep
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bw.q4_moe(x, idx, wts, *handles, stream=side)
    side.synchronize()
    assert torch.equal(got, y)


def test_empty_calls():
    note("[moe] no tokens")
    handles = [bw.q4_upload(*(cuda(v) for v in w)) for w in experts(80, 2, 128, 128, 128, False)]
    idx, w = bw.moe_route(torch.empty((0, 2), device="cuda"), 1)
    assert idx.shape == w.shape == (0, 1)
    assert bw.moe_route_backward(torch.empty((0, 2), device="cuda"), idx, w).shape == (0, 2)
    assert bw.q4_moe(torch.empty((0, 128), device="cuda"), idx, w, *handles).shape == (0, 128)
