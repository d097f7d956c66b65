"""GPU parity of a whole mixture-of-experts layer with a 64-bit reference.

Chosen experts are compared as whole numbers: rows are normed from f64 statistics, logits are f64 sums rounded to f32, and
the reference does the same (two f64 sums of one value are 2^-45 of their terms apart, which moves an f32 logit once in 2^20
and a decision only where two keys are as close).  Weights: (span + 12) 2^-23 of the weight, as the router's.  The rows: the
result's rounding, half a step of y; silu(g) u's rounding to f16, 2^-11 of the experts' part in the norm of a row, and f32 sums, 2^-18.
"""

import math
import warnings

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import half_step, layer64
from gpu_util import note
from q4_util import DTYPES, cuda, gen, weight

pytestmark = pytest.mark.gpu


def inputs(t, e, d, f, group, zeros, dtype, norm="own", router="f32", bias=False, residual=True, seed=1):
    ty = DTYPES[dtype]
    g = gen(seed)
    side = lambda kind: ty if kind == "own" else DTYPES[kind]  # noqa: E731
    w = [weight(seed + 1, (e,), f, d, group, zeros), weight(seed + 2, (e,), f, d, group, zeros), weight(seed + 3, (e,), d, f, group, zeros)]
    x = ((3.0 if norm else 1.0) * torch.randn((t, d), generator=g)).to(ty)
    a = dict(norm=(1 + 0.1 * torch.randn(d, generator=g)).to(side(norm)) if norm else None,
             bias=0.1 * torch.randn(e, generator=g) if bias else None,
             residual=torch.randn((t, d), generator=g).to(ty) if residual else None)
    r = (torch.randn((e, d), generator=g) / math.sqrt(d)).to(side(router))
    return x, r, w, a


def call(x, r, handles, k, a, **kw):
    return bw.moe_layer(x.cuda(), r.cuda(), *handles, k, **{n: cuda(v) for n, v in a.items()}, **kw)


def check(x, r, w, k, a, dtype, what, **kw):
    t, d = x.shape
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    ty = DTYPES[dtype]
    by = torch.full((t * d + 64,), float("nan"), dtype=ty, device="cuda")
    bi = torch.full((t * k + 8,), -77, dtype=torch.int32, device="cuda")
    bo = torch.full((t * k + 8,), float("nan"), device="cuda")
    note(f"[moe_layer {what}] T={t} E={r.shape[0]} k={k} d={d} f={w[0][0].shape[1]} {dtype} router={r.dtype} {kw}")
    y, idx, wts = call(x, r, handles, k, a, y=by[: t * d].view(t, d), idx=bi[: t * k].view(t, k), weights=bo[: t * k].view(t, k), **kw)
    torch.cuda.synchronize()
    assert torch.isnan(by[t * d:]).all() and (bi[t * k:] == -77).all() and torch.isnan(bo[t * k:]).all(), "write past the end"
    part, want_i, want_w, logits = layer64(x, r, *w, k, **a, **kw)
    assert torch.equal(idx.cpu(), want_i), what
    fin = logits[torch.isfinite(logits)].double()
    span = float((fin.max() - fin.min()).clamp(min=fin.abs().max()))
    assert ((wts.cpu().double() - want_w).abs() <= (span + 12) * 2.0 ** -23 * want_w + 2.0 ** -149).all(), what
    want = part if a["residual"] is None else part + a["residual"].double()
    err = (y.cpu().double() - want).norm(dim=1)
    tol = (2.0 ** -18 + (0 if dtype == "f32" else 2.0 ** -11)) * part.norm(dim=1) + half_step(dtype) * want.norm(dim=1) * 1.01 + 1e-30
    note(f"  worst row {float((err / tol).max()):.3g} of the tolerance")
    assert (err <= tol).all(), what
    again = call(x, r, handles, k, a, **kw)
    assert all(torch.equal(p, q) for p, q in zip((y, idx, wts), again)), "not deterministic"
    return y, idx, wts


ROUTERS = {"softmax": dict(), "renorm": dict(renorm=True), "sigmoid": dict(score="sigmoid", renorm=True),
           "groups": dict(score="sigmoid", groups=4, keep=2, group_top=2, renorm=True), "best": dict(groups=4, keep=3)}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("router", list(ROUTERS))
@pytest.mark.parametrize("t,e,k,d,f,group,zeros", [(1, 4, 1, 128, 128, 128, False), (1, 64, 8, 512, 256, 64, True),
                                                   (3, 16, 4, 288, 96, 32, True), (8, 64, 6, 256, 128, 128, False),
                                                   (20, 8, 2, 256, 192, 64, True), (70, 32, 4, 256, 128, 128, False),
                                                   (300, 8, 2, 384, 256, 32, True)])
def test_layer(t, e, k, d, f, group, zeros, router, dtype):
    bias = router == "groups"
    x, r, w, a = inputs(t, e, d, f, group, zeros, dtype, norm="own" if t % 2 else "f32", router="f32" if t > 2 else "own", bias=bias)
    check(x, r, w, k, a, dtype, router, **ROUTERS[router])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 2, 9, 40, 130])
@pytest.mark.parametrize("norm,residual,bias", [(None, False, False), (None, True, True), ("own", False, True)])
def test_parts(norm, residual, bias, t, dtype):
    x, r, w, a = inputs(t, 16, 256, 128, 64, False, dtype, norm=norm, residual=residual, bias=bias)
    check(x, r, w, 2, a, dtype, f"norm={norm} residual={residual} bias={bias}")


@pytest.mark.parametrize("t", [1, 5, 64])
@pytest.mark.parametrize("e,k,d", [(1, 1, 128), (3, 3, 2080), (65, 7, 160), (130, 64, 128), (1024, 8, 64)])
def test_numbers_of_experts(e, k, d, t):
    x, r, w, a = inputs(t, e, d, 64, 32, False, "bf16")
    check(x, r, w, k, a, "bf16", "experts", renorm=True)


def test_more_tokens_than_a_grids_axis():
    """70000 tokens: every choice against torch's f64 product, some rows of the result against the reference."""
    t, e, k, d = 70000, 4, 1, 64
    x, r, w, a = inputs(t, e, d, 32, 32, False, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    note(f"[moe_layer] T={t}")
    y, idx, _ = call(x, r, handles, k, a)
    v = x.cuda().double()
    n = (v / ((v * v).mean(1, keepdim=True) + 1e-6).sqrt() * a["norm"].cuda().double()).bfloat16()
    logits = (n.double() @ r.cuda().double().T.contiguous()).float()
    top = logits.topk(2, 1).values
    clear = top[:, 0] - top[:, 1] > 2.0 ** -10  # (a row whose roundings differ moves its logits by less)
    assert torch.equal(idx[clear, 0].long(), logits.argmax(1)[clear])
    some = torch.cat((torch.arange(5), torch.arange(65530, 65545), torch.arange(t - 5, t)))
    part, want_i, _, _ = layer64(x[some], r, *w, k, norm=a["norm"])
    want = part + a["residual"][some].double()
    assert torch.equal(idx[some.cuda()].cpu(), want_i)
    err = (y[some.cuda()].cpu().double() - want).norm(dim=1)
    assert (err <= (2.0 ** -18 + 2.0 ** -11) * part.norm(dim=1) + half_step("bf16") * want.norm(dim=1) * 1.01).all()


@pytest.mark.parametrize("t", [1, 7, 200])
def test_masked_experts_and_tokens_without_one(t):
    """Biases of -inf mask experts; where fewer are left than slots these are -1, and a token without any gets its residual."""
    x, r, w, a = inputs(t, 8, 128, 128, 64, False, "bf16", bias=True)
    a["bias"][2:] = -math.inf
    _, idx, wts = check(x, r, w, 4, a, "bf16", "masks", score="sigmoid", renorm=True)
    assert (idx[:, 2:] == -1).all() and (wts[:, 2:] == 0).all()
    a["bias"][:] = -math.inf
    y, idx, _ = check(x, r, w, 4, a, "bf16", "all masked", score="softmax")
    assert (idx == -1).all() and torch.equal(y.cpu(), a["residual"])


@pytest.mark.parametrize("t", [1, 4, 100])
def test_equal_logits_take_the_lower_index(t):
    x, r, w, a = inputs(t, 12, 128, 128, 64, False, "f32")
    r[:] = r[0]
    _, idx, _ = check(x, r, w, 3, a, "f32", "ties")
    assert (idx.cpu() == torch.tensor([0, 1, 2])).all()


@pytest.mark.parametrize("t", [1, 6, 90])
def test_a_nan_row_stays_alone(t):
    x, r, w, a = inputs(t, 8, 128, 128, 64, False, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    clean = call(x, r, handles, 2, a)
    x[t // 2, 3] = float("nan")
    note(f"[moe_layer] NaN row T={t}")
    y, idx, wts = call(x, r, handles, 2, a)
    torch.cuda.synchronize()
    rest = [i for i in range(t) if i != t // 2]
    assert torch.isnan(y[t // 2]).all()
    assert all(torch.equal(p[rest], q[rest]) for p, q in zip((y, idx, wts), clean))


@pytest.mark.parametrize("t", [1, 8, 150])
def test_in_place_of_the_residual(t):
    x, r, w, a = inputs(t, 16, 256, 128, 128, False, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    note(f"[moe_layer] in place T={t}")
    want, _, _ = call(x, r, handles, 2, a)
    y = cuda(a["residual"]).clone()
    got, _, _ = bw.moe_layer(x.cuda(), r.cuda(), *handles, 2, norm=cuda(a["norm"]), residual=y, y=y)
    assert got is y and torch.equal(got, want)
    # the residual that is x itself
    xs = x.cuda()
    got, _, _ = bw.moe_layer(xs, r.cuda(), *handles, 2, norm=cuda(a["norm"]), residual=xs)
    want, _, _ = call(x, r, handles, 2, dict(a, residual=x))
    assert torch.equal(got, want)


@pytest.mark.parametrize("t", [1, 8, 40, 300])
def test_in_a_graph_and_on_another_stream(t):
    x, r, w, a = inputs(t, 16, 256, 128, 64, True, "bf16", bias=True)
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    x, r, a = x.cuda(), r.cuda(), {k: cuda(v) for k, v in a.items()}
    kw = dict(a, score="sigmoid", renorm=True)
    note(f"[moe_layer] graph T={t}")
    bw.moe_layer(x, r, *handles, 4, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bw.moe_layer(x, r, *handles, 4, **kw)
    for rep in range(5):
        x.copy_(torch.randn(x.shape, generator=gen(20 + rep)).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        want = bw.moe_layer(x, r, *handles, 4, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), rep
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = bw.moe_layer(x, r, *handles, 4, **kw, stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(there, want))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 5])
def test_workgroups_that_form_what_they_wait_for(t, dtype):
    """With no patience every down workgroup may find silu(g) u missing and form it itself: the same bits."""
    x, r, w, a = inputs(t, 16, 256, 192, 64, True, dtype)
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    note(f"[moe_layer] no patience T={t} {dtype}")
    want = call(x, r, handles, 3, a)
    torch.cuda.synchronize()
    was = bw.moe_layer_set_patience(0)
    try:
        for _ in range(5):
            got = call(x, r, handles, 3, a)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))
    finally:
        assert bw.moe_layer_set_patience(was) == 0
    with pytest.raises(bw.Tq2Error):
        bw.moe_layer_set_patience(-1)


def test_calls_side_by_side():
    """Many calls on two streams at once, each with a workspace of its own."""
    x, r, w, a = inputs(8, 16, 256, 128, 64, True, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    x, r, a = x.cuda(), r.cuda(), {k: cuda(v) for k, v in a.items()}
    rows = [x[i: i + n].contiguous() for i, n in ((0, 1), (1, 1), (0, 8), (3, 5))]
    res = [a["residual"][i: i + n].contiguous() for i, n in ((0, 1), (1, 1), (0, 8), (3, 5))]
    one = lambda i, s=None: bw.moe_layer(rows[i], r, *handles, 4, norm=a["norm"], residual=res[i], stream=s)  # noqa: E731
    want = [one(i) for i in range(4)]
    torch.cuda.synchronize()
    note("[moe_layer] two streams")
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(i % 4, one(i % 4, streams[i % 3])) for i in range(48)]
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))


def test_a_block_of_all_operators():
    """Linear, norms and layer one after another, as a block of a model runs them, against its formula in f64."""
    t, d, e, k = 24, 256, 8, 2
    x, r, w, a = inputs(t, e, d, 128, 64, False, "f32", norm=None, residual=False)
    proj = weight(40, (), d, d, 64, True)
    post, pre = (1 + 0.1 * torch.randn(d, generator=gen(i)) for i in (41, 42))
    bias, gate = 0.1 * torch.randn(d, generator=gen(43)), 0.5 + 0.2 * torch.randn((1, d), generator=gen(44))
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    h = bw.q4_upload(*(cuda(v) for v in proj))
    note("[block] all operators")
    b = bw.q4_linear(h, x.cuda(), bias=bias.cuda(), activation="silu")
    y, n = bw.block_norm(x.cuda(), b=b, post=post.cuda(), gate=gate.cuda(), scale=0.5, pre=pre.cuda())
    out, idx, wts = bw.moe_layer(n, r.cuda(), *handles, k, residual=y, renorm=True)
    from block_util import norm64
    from q4_util import dequant64
    z = x.double() @ dequant64(*proj).T + bias.double()
    y64 = x.double() + 0.5 * gate.double() * norm64(z * torch.sigmoid(z), "rms", 1e-6, post.double(), None)
    assert float((y.cpu().double() - y64).norm() / y64.norm()) <= 2.0 ** -18
    n64 = norm64(y64, "rms", 1e-6, pre.double(), None)
    assert float((n.cpu().double() - n64).norm() / n64.norm()) <= 2.0 ** -18
    part, want_i, _, _ = layer64(n.cpu(), r, *w, k, renorm=True)  # the choice follows the rows as they are
    assert torch.equal(idx.cpu(), want_i)
    assert float((out.cpu().double() - y64 - part).norm() / (y64 + part).norm()) <= 2.0 ** -17


def test_refusals_and_empty_calls():
    x, r, w, a = inputs(6, 8, 128, 64, 32, False, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    x, r, a = x.cuda(), r.cuda(), {k: cuda(v) for k, v in a.items()}
    note("[moe_layer] refusals")
    f = lambda **kw: bw.moe_layer(**dict(dict(x=x, router=r, gate=handles[0], up=handles[1], down=handles[2], k=2), **kw))  # noqa: E731
    for bad in (dict(k=0), dict(k=9), dict(x=x[:, :64].contiguous()), dict(router=r[:7]), dict(norm=r[0, :64].contiguous()), dict(groups=3),
                dict(groups=4, keep=5), dict(group_top=3), dict(score="relu"), dict(bias=torch.zeros(7, device="cuda")),
                dict(residual=x[:5]), dict(y=x[:5]), dict(up=handles[2]), dict(x=x[0]),
                dict(idx=torch.zeros((6, 3), dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            f(**bad)
    for bad in (dict(router=r.half()), dict(router=None), dict(x=x.double()), dict(norm=r[0].half()), dict(bias=r[0, :8].bfloat16()),
                dict(residual=x.float()), dict(idx=torch.zeros((6, 2), device="cuda")), dict(k="2")):
        with pytest.raises(TypeError):
            f(**bad)
    with pytest.raises(bw.Tq2Error):
        f(y=x)
    with pytest.raises(bw.Tq2Error):
        f(residual=x, y=x)
    y, idx, wts = f(x=x[:0], residual=x[:0])
    assert y.shape == (0, 128) and idx.shape == wts.shape == (0, 2)
    with pytest.warns(UserWarning, match="moe_layer forms no gradients"):
        f(router=r.clone().requires_grad_())
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        f(x=x.clone().requires_grad_())
