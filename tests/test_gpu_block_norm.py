"""GPU parity of a block's norms and their gradient with 64-bit references.

Tolerances, element by element.  Forward: statistics and normed values come from f64 and are rounded to f32 once (2^-24); y is
three f32 operations on scale, gate and u and one on x: 4 2^-24 of the terms' size, then half a step of its type.  n is
compared as the norm of the kernel's own y: 2^-24 and half a step.
Gradient: every sum over a row is f32's over at most 16 terms a thread, then a tree over at most 1024 threads: 32 roundings, and
its terms have eight more; so 64 2^-24 of the sum of the magnitudes of what a formula adds, A for dx, and the same again on what
depends on dx.  Sums over rows: M 2^-24 more of theirs.  Then half a step for dx and db.
"""

import warnings

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import d64, half_step, hat64, least, norm64, u64
from gpu_util import note
from q4_util import DTYPES, gen

pytestmark = pytest.mark.gpu
EPS = 1e-6


def inputs(m, n, dtype, kind, post, pre, gates, wide=False, seed=1, offset=0.0):
    t = DTYPES[dtype]
    wt = torch.float32 if wide else t
    g = gen(seed)
    rand = lambda *s, about=0.0, width=1.0, to=t: (about + width * torch.randn(s, generator=g)).to(to).cuda()  # noqa: E731
    a = dict(x=rand(m, n, about=offset, width=2.0), b=rand(m, n, about=offset))
    a["gate"] = rand(gates, n, about=0.5, width=0.3, to=wt) if gates else None
    for name, on in (("post", post), ("pre", pre)):
        a[name] = rand(n, about=1.0, width=0.1, to=wt) if on else None
        a[name + "_bias"] = rand(n, width=0.1, to=wt) if on and kind == "layer" else None
    return a


def guarded(m, n, t):
    base = torch.full((m * n + 64,), float("nan"), dtype=t, device="cuda")
    return base, base[: m * n].view(m, n)


def check_forward(a, m, n, dtype, kind, scale, eps=EPS):
    t = DTYPES[dtype]
    by, y = guarded(m, n, t)
    bn, nn = guarded(m, n, t)
    pre = a["pre"] is not None
    gy, gn = bw.block_norm(a["x"], b=a["b"], post=a["post"], post_bias=a["post_bias"], gate=a["gate"], scale=scale, pre=a["pre"],
                           pre_bias=a["pre_bias"], kind=kind, eps=eps, y=y, n=nn if pre else None)
    torch.cuda.synchronize()
    assert torch.isnan(by[m * n:]).all() and torch.isnan(bn[m * n:]).all(), "write past the end"
    assert gy is y and (gn is nn if pre else gn is None)
    w = {k: d64(v) for k, v in a.items()}
    u = u64(w["b"], w["post"], w["post_bias"], kind, eps)
    gate = 1.0 if w["gate"] is None else w["gate"].repeat_interleave(m // w["gate"].shape[0], 0)
    add = scale * gate * u
    want = w["x"] + add
    tol = 4 * 2.0 ** -24 * (add.abs() + w["x"].abs()) + half_step(dtype) * want.abs() * 1.01 + least(dtype)
    err = (y.double() - want).abs()
    note(f"  y worst err/tol {float((err / tol).max()):.3g}")
    assert (err <= tol).all()
    if pre:
        want = norm64(y.double(), kind, eps, w["pre"], w["pre_bias"])
        tol = (2.0 ** -23 + half_step(dtype)) * want.abs() + 2.0 ** -40 + least(dtype)
        err = (nn.double() - want).abs()
        note(f"  n worst err/tol {float((err / tol).max()):.3g}")
        assert (err <= tol).all()
    return y


def check_backward(a, y, m, n, dtype, kind, scale, eps=EPS, dy_given=True, seed=50):
    t = DTYPES[dtype]
    pre, post, has_b, gates = a["pre"] is not None, a["post"] is not None, a["b"] is not None, a["gate"] is not None
    dy = (0.5 * torch.randn((m, n), generator=gen(seed))).to(t).cuda() if dy_given else None
    dn = (0.5 * torch.randn((m, n), generator=gen(seed + 1))).to(t).cuda() if pre else None
    bx, dx = guarded(m, n, t)
    bb, db = guarded(m, n, t)
    out = bw.block_norm_backward(dy, y, dn=dn, b=a["b"], post=a["post"], post_bias=a["post_bias"], gate=a["gate"], scale=scale,
                                 pre=a["pre"], pre_bias=a["pre_bias"], kind=kind, eps=eps, dx=dx, db=db if has_b else None)
    torch.cuda.synchronize()
    assert torch.isnan(bx[m * n:]).all() and torch.isnan(bb[m * n:]).all(), "write past the end"
    w = {k: d64(v) for k, v in a.items()}
    dY = torch.zeros((m, n), dtype=torch.float64, device="cuda") if dy is None else dy.double()
    A, step, tol = dY.abs(), 2.0 ** -24, {}
    want, mean = {}, lambda v: v.mean(1, keepdim=True)

    def back(g, v):
        """Through a norm: the gradient, and the sum of the magnitudes of its terms."""
        hat = hat64(v, kind, eps)
        c = v - mean(v) if kind == "layer" else v
        rstd = 1 / (mean(c * c) + eps).sqrt()
        d = (g - hat * mean(g * hat) - (mean(g) if kind == "layer" else 0.0)) * rstd
        return d, hat, rstd

    if pre:
        g = dn.double() * w["pre"]
        d, hat, rstd = back(g, y.double())
        dY = dY + d
        A = A + (g.abs() + mean(g.abs()) + hat.abs() * mean((g * hat).abs())) * rstd
        want["dpre"], tol["dpre"] = (dn.double() * hat).sum(0), (m + 64) * step * (dn.double() * hat).abs().sum(0)
        if a["pre_bias"] is not None:
            want["dpre_bias"], tol["dpre_bias"] = dn.double().sum(0), (m + 64) * step * dn.double().abs().sum(0)
    want["dx"], tol["dx"] = dY, 64 * step * A + half_step(dtype) * dY.abs() * 1.01 + least(dtype)
    if has_b:
        gate = torch.ones_like(dY) if not gates else w["gate"].repeat_interleave(m // w["gate"].shape[0], 0)
        u = u64(w["b"], w["post"], w["post_bias"], kind, eps)
        du, B = scale * gate * dY, (scale * gate).abs() * A
        if gates:
            by = lambda v: v.view(w["gate"].shape[0], -1, n).sum(1)  # noqa: E731
            want["dgate"] = scale * by(u * dY)
            terms = u.abs() + (0 if a["post_bias"] is None else 2 * w["post_bias"].abs())
            tol["dgate"] = (m + 128) * step * abs(scale) * by(terms * A)
        if post:
            d, hat, rstd = back(du * w["post"], w["b"])
            Bw = B * w["post"].abs()
            want["db"] = d
            tol["db"] = 128 * step * (Bw + mean(Bw) + hat.abs() * mean(Bw * hat.abs())) * rstd
            want["dpost"], tol["dpost"] = (du * hat).sum(0), (m + 128) * step * (B * hat.abs()).sum(0)
            if a["post_bias"] is not None:
                want["dpost_bias"], tol["dpost_bias"] = du.sum(0), (m + 128) * step * B.sum(0)
        else:
            want["db"], tol["db"] = du, 72 * step * B
        tol["db"] = tol["db"] + half_step(dtype) * want["db"].abs() * 1.01 + least(dtype)
    assert set(out) == set(want)
    for name, v in want.items():
        assert out[name].dtype == (t if name in ("dx", "db") else torch.float32) and out[name].shape == v.shape, name
        err, bound = (out[name].double() - v).abs(), tol[name] + 1e-42
        note(f"  {name} worst err/tol {float((err / bound).max()):.3g}")
        assert (err <= bound).all(), name
    return out


SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (4, 9), (9, 63), (130, 64), (33, 100), (6, 513), (300, 512), (17, 1111), (70, 2048),
         (8, 2050), (12, 4096), (5, 4100), (3, 8192), (2, 9001), (2, 16384)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("m,n", SIZES)
def test_sizes(m, n, kind, dtype):
    note(f"[block_norm] M={m} N={n} {kind} {dtype}")
    a = inputs(m, n, dtype, kind, True, True, 1)
    y = check_forward(a, m, n, dtype, kind, 0.7)
    check_backward(a, y, m, n, dtype, kind, 0.7)


@pytest.mark.parametrize("dtype,wide", [("bf16", True), ("bf16", False), ("f16", True), ("f32", True)])
@pytest.mark.parametrize("m,gates", [(12, 1), (12, 12), (12, 3), (600, 2), (600, 600), (602, 7), (1030, 515)])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_parts_and_gates(post, pre, m, gates, dtype, wide):
    n, kind = 264, "layer" if m == 602 else "rms"
    note(f"[block_norm] M={m} gates={gates} post={post} pre={pre} {dtype} wide={wide}")
    a = inputs(m, n, dtype, kind, post, pre, gates, wide)
    y = check_forward(a, m, n, dtype, kind, 1.0)
    check_backward(a, y, m, n, dtype, kind, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_one_norm_alone(kind, dtype):
    """Without a block: n from x, and its gradient with and without one for x itself."""
    m, n = 37, 1000
    a = inputs(m, n, dtype, kind, False, True, 0)
    x = a["x"]
    note(f"[block_norm] norm alone {kind} {dtype}")
    y, nn = bw.block_norm(x, pre=a["pre"], pre_bias=a["pre_bias"], kind=kind)
    assert y is x
    want = norm64(x.double(), kind, EPS, a["pre"].double(), d64(a["pre_bias"]))
    assert ((nn.double() - want).abs() <= (2.0 ** -23 + half_step(dtype)) * want.abs() + 2.0 ** -40).all()
    a.update(b=None)
    for dy_given in (True, False):
        check_backward(a, x, m, n, dtype, kind, 1.0, dy_given=dy_given)


def test_no_gate():
    a = inputs(50, 300, "f32", "rms", True, True, 0)
    note("[block_norm] no gate")
    y = check_forward(a, 50, 300, "f32", "rms", 0.3)
    check_backward(a, y, 50, 300, "f32", "rms", 0.3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_biases_without_means(post, pre, dtype):
    m, n = 20, 520
    a = inputs(m, n, dtype, "layer", post, pre, 1)
    note(f"[block_norm] rms with biases post={post} pre={pre} {dtype}")
    y = check_forward(a, m, n, dtype, "rms", 0.8)
    check_backward(a, y, m, n, dtype, "rms", 0.8)
    for name in ("post_bias", "pre_bias"):  # one of the two
        one = dict(a, **{name: None})
        check_backward(one, check_forward(one, m, n, dtype, "rms", 0.8), m, n, dtype, "rms", 0.8)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_far_from_zero_and_of_any_size(kind):
    """A mean 2000 times the deviation, rows of 1e30 and 1e-30, constant rows and rows of zeros."""
    m, n = 12, 500
    a = inputs(m, n, "f32", kind, True, True, 1, offset=2000.0)
    for v in (a["x"], a["b"]):
        v[1] = 0
        v[2] = 3.5
        v[3] = 1e30 * (v[3] - 2000)
        v[4] = 1e-30 * (v[4] - 2000)
    a["x"][6] = -a["b"][6]
    note(f"[block_norm] far rows {kind}")
    check_forward(a, m, n, "f32", kind, 1.0, eps=1e-5)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradient_against_differences(kind):
    """The kernel's gradient against central differences of the f64 forward (step 1e-5, error below 1e-8) along random directions."""
    m, n, scale = 6, 40, 0.6
    a = inputs(m, n, "f32", kind, True, True, 2)
    y, _ = bw.block_norm(a["x"], b=a["b"], post=a["post"], post_bias=a["post_bias"], gate=a["gate"], scale=scale, pre=a["pre"],
                         pre_bias=a["pre_bias"], kind=kind)
    dy, dn = (torch.randn((m, n), generator=gen(i)).cuda() for i in (60, 61))
    note(f"[block_norm_backward] differences {kind}")
    out = bw.block_norm_backward(dy, y, dn=dn, b=a["b"], post=a["post"], post_bias=a["post_bias"], gate=a["gate"], scale=scale,
                                 pre=a["pre"], pre_bias=a["pre_bias"], kind=kind)
    w = {k: d64(v) for k, v in a.items() if v is not None}

    def loss(w):
        u = norm64(w["b"], kind, EPS, w["post"], w.get("post_bias"))
        yy = w["x"] + scale * w["gate"].repeat_interleave(m // 2, 0) * u
        return float((dy.double() * yy).sum() + (dn.double() * norm64(yy, kind, EPS, w["pre"], w.get("pre_bias"))).sum())

    for name in w:
        for i in range(3):
            d = torch.randn(w[name].shape, generator=gen(70 + i), dtype=torch.float64).cuda()
            diff = (loss(dict(w, **{name: w[name] + 1e-5 * d})) - loss(dict(w, **{name: w[name] - 1e-5 * d}))) / 2e-5
            got = float((out["d" + name].double() * d).sum())
            size = float((out["d" + name].double() * d).abs().sum())
            # y was rounded to f32: 2^-24 of what it changes in the second norm's gradient
            assert abs(diff - got) <= 1e-6 + 256 * 2.0 ** -24 * size, (name, diff, got)


def test_nan_and_infinite_rows_stay_apart():
    m, n = 40, 1000
    a = inputs(m, n, "bf16", "rms", True, True, 1)
    call = lambda: bw.block_norm(a["x"], b=a["b"], post=a["post"], gate=a["gate"], pre=a["pre"])  # noqa: E731
    clean = call()
    a["b"][3, 5], a["x"][7, 999] = float("nan"), float("inf")
    note("[block_norm] NaN rows")
    rest = [i for i in range(m) if i not in (3, 7)]
    for got, was in zip(call(), clean):
        assert torch.equal(got[rest], was[rest]) and torch.isnan(got[3]).all()


@pytest.mark.parametrize("m,n,gates", [(3, 512, 1), (700, 1000, 7)])
def test_in_a_graph_and_on_another_stream(m, n, gates):
    a = inputs(m, n, "bf16", "layer", True, True, gates)
    dy, dn = (torch.randn((m, n), generator=gen(i)).bfloat16().cuda() for i in (80, 81))
    kw = dict(post=a["post"], post_bias=a["post_bias"], gate=a["gate"], scale=0.5, pre=a["pre"], pre_bias=a["pre_bias"], kind="layer")

    def work(**more):
        y, nn = bw.block_norm(a["x"], b=a["b"], **kw, **more)
        return [y, nn, *bw.block_norm_backward(dy, y, dn=dn, b=a["b"], **kw, **more).values()]

    note(f"[block_norm] graph M={m} N={n}")
    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for rep in range(4):
        a["b"].copy_(torch.randn((m, n), generator=gen(90 + rep)))
        dn.copy_(torch.randn((m, n), generator=gen(95 + rep)))
        graph.replay()
        torch.cuda.synchronize()
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), rep
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    there = work(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(there, want))


def test_refusals_and_empty_calls():
    m, n = 6, 64
    a = inputs(m, n, "bf16", "layer", True, True, 1)
    x, b, post, gate, pre = (a[k] for k in ("x", "b", "post", "gate", "pre"))
    note("[block_norm] refusals")
    for bad in (dict(), dict(post=post, pre=pre), dict(b=b, post_bias=post), dict(b=b, pre_bias=pre), dict(gate=gate, pre=pre),
                dict(b=b[:5]), dict(b=b, gate=gate[0]), dict(b=b, gate=torch.ones((4, n), dtype=x.dtype, device="cuda")),
                dict(b=b, post=post[:63]), dict(b=b, kind="batch"), dict(pre=pre, y=torch.empty_like(x)),
                dict(b=b, n=torch.empty_like(x)), dict(b=b.T.contiguous().T)):
        with pytest.raises(ValueError):
            bw.block_norm(x, **bad)
    for bad in (dict(b=b.float()), dict(b=b, post=post.half()), dict(b=b, post=post.float(), pre=pre), dict(b=b, scale="1")):
        with pytest.raises(TypeError):
            bw.block_norm(x, **bad)
    with pytest.raises(ValueError):
        bw.block_norm(torch.zeros((2, 16385), device="cuda"), pre=torch.zeros(16385, device="cuda"))
    for bad in (dict(b=b, y=x), dict(b=b, y=b), dict(b=b, pre=pre, y=(t := torch.empty_like(x)), n=t)):
        with pytest.raises(bw.Tq2Error):
            bw.block_norm(x, **bad)
    for args in ((None, x), (x, x, None, None, post), (x, None, x, None, None, None, None, 1.0, pre), (x, x, x), (x, x, None, None, None, None, gate)):
        with pytest.raises(ValueError):
            bw.block_norm_backward(*args)
    with pytest.raises(bw.Tq2Error):
        bw.block_norm_backward(x, x, dn=b, pre=pre, dx=x)
    y, nn = bw.block_norm(x[:0], b=b[:0], post=post, gate=gate, pre=pre)
    assert y.shape == nn.shape == (0, n)
    out = bw.block_norm_backward(x[:0], y, dn=nn, b=b[:0], post=post, gate=gate, pre=pre)
    assert out["dx"].shape == (0, n) and all((out[k] == 0).all() for k in ("dgate", "dpost", "dpre")), "sums over no rows"
    with pytest.warns(UserWarning, match="block_norm records no gradient"):
        bw.block_norm(x, pre=pre.clone().requires_grad_())
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        bw.block_norm(x.clone().requires_grad_(), b=b, pre=pre)
