"""Refusals and sizes of the block's calls (no GPU needed), and their 64-bit references pinned to closed forms."""

import math

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import CODES, LayerCall, NormBackwardCall, NormCall, act64, hat64
from test_q4_cpu import A, L, ptr, w4  # noqa: F401  (L: the fixture)

BAD = bw.TQ2_EINVAL
AT = [A + (i << 24) for i in range(24)]
PAST_THE_CHECKS = (bw.TQ2_ENODEV, bw.TQ2_EDEVICE)  # the arguments pass; there is no gfx950 here


def test_linear_refusals(L):
    w = w4(data=AT[0])
    x, b, r, y = AT[1:5]

    def call(w=w, x=x, bias=b, btype=0, act=0, r=r, y=y, m=4, dtype=2, ws=None, nws=0):
        return L.q4_linear(ptr(w) if w is not None else None, x, bias, btype, act, r, y, m, dtype, ws, nws, None)

    if not torch.cuda.is_available():
        for ok in (dict(), dict(bias=None, btype=7), dict(r=None), dict(btype=2), dict(r=y), dict(act=4), dict(m=0), dict(r=x)):
            assert call(**ok) in PAST_THE_CHECKS, ok
    for bad in (dict(w=None), dict(w=w4(e=2, data=AT[0])), dict(x=None), dict(y=None), dict(act=5), dict(act=-1), dict(btype=1), dict(btype=3),
                dict(dtype=3), dict(m=-1), dict(m=1 << 31), dict(x=x + 8), dict(y=y + 8), dict(r=r + 8), dict(bias=b + 2), dict(y=x),
                dict(y=AT[0]), dict(y=b - 16), dict(r=y + 16), dict(r=y - 16)):
        assert call(**bad) == BAD, bad
    big = w4(n=4096, k=4096, g=128, data=AT[0])
    need = L.q4_gemm_workspace_size(ptr(big), 2048, 2)
    far = A + (1 << 30)
    kw = dict(w=big, m=2048, x=AT[2], y=AT[6], r=AT[10], bias=AT[14])
    for ws in (AT[2], AT[6], AT[10], AT[14], AT[0], AT[10] - need + 256, far + 8, None):
        assert call(**kw, ws=ws, nws=need) == BAD, ws
    assert call(**kw, ws=far, nws=need - 1) == BAD


def held(f, c, *args):
    """f(address of c, ...) while c lives."""
    return f(ptr(c), *args)


def layer_call(g, u, d, **kw):
    c = LayerCall(x=AT[3], norm=AT[4], router=AT[5], bias=AT[6], gate=ptr(g), up=ptr(u), down=ptr(d), residual=AT[7], y=AT[8],
                  idx=AT[9], weights=AT[10], eps=1e-6, T=5, k=2, groups=1, keep=1, group_top=1, score=0, renorm=1, dtype=2, norm_dtype=0,
                  router_dtype=0)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def test_layer_refusals(L):
    gate, up, down = w4(4, 64, 128, data=AT[0]), w4(4, 64, 128, data=AT[1]), w4(4, 128, 64, data=AT[2])
    other = w4(4, 64, 128, g=64, data=AT[1])
    need = L.moe_layer_workspace_size(5, 2, 4, 128, 64, 2, 1)
    ws = AT[12]

    def call(at=ws, size=need, **kw):
        return held(L.moe_layer, layer_call(gate, up, down, **kw), at, size, None)

    if not torch.cuda.is_available():
        for ok in (dict(), dict(norm=None), dict(bias=None), dict(residual=None), dict(residual=AT[8]), dict(residual=AT[3]), dict(T=0),
                   dict(router_dtype=2), dict(score=1, groups=2, keep=1, group_top=2)):
            assert call(**ok) in PAST_THE_CHECKS, ok
    for bad in (dict(x=None), dict(router=None), dict(y=None), dict(idx=None), dict(weights=None), dict(gate=None), dict(up=ptr(other)),
                dict(down=ptr(gate)), dict(T=-1), dict(k=0), dict(k=5), dict(groups=3), dict(groups=0), dict(keep=2), dict(group_top=3),
                dict(score=2), dict(dtype=3), dict(router_dtype=1), dict(norm_dtype=1), dict(x=AT[3] + 8), dict(y=AT[8] + 4),
                dict(router=AT[5] + 4), dict(norm=AT[4] + 2), dict(idx=AT[9] + 2), dict(y=AT[3]), dict(y=AT[0]), dict(y=AT[5]), dict(idx=AT[8]),
                dict(weights=AT[9]), dict(idx=AT[7]), dict(residual=AT[8] + 16), dict(weights=AT[6]), dict(idx=AT[4])):
        assert call(**bad) == BAD, bad
    for at in (*AT[:11], AT[3] - need + 256, ws + 16, None):
        assert call(at=at) == BAD, at
    assert call(size=need - 1) == BAD and L.moe_layer(None, ws, need, None) == BAD


def test_layer_workspace_sizes(L):
    for t in (0, 1, 8, 300):
        for dtype in (0, 1, 2):
            with_norm, without = (L.moe_layer_workspace_size(t, 2, 8, 256, 128, dtype, n) for n in (1, 0))
            assert 0 < without <= with_norm
            assert with_norm >= L.q4_moe_workspace_size(t, 2, 8, 256, 128, dtype)
    for bad in ((-1, 2, 8, 256, 128, 0), (1, 0, 8, 256, 128, 0), (1, 9, 8, 256, 128, 0), (1, 2, 0, 256, 128, 0), (1, 2, 8, 250, 128, 0),
                (1, 2, 8, 256, 0, 0), (1, 2, 8, 256, 128, 3), (1 << 24, 2, 8, 256, 128, 0)):
        assert L.moe_layer_workspace_size(*bad, 1) == 0, bad


def norm_call(cls, **kw):
    names = [f[0] for f in cls._fields_]
    names = names[: names.index("eps")]
    c = cls(**{n: AT[i] for i, n in enumerate(names)}, eps=1e-6, M=6, N=64, R=2, scale=1.0, layer=1, dtype=2, weights_dtype=0)
    for n, v in kw.items():
        setattr(c, n, v)
    return c


def test_block_norm_refusals(L):
    call = lambda **kw: held(L.block_norm, norm_call(NormCall, **kw), None)  # noqa: E731
    x, b, post, post_bias, gate, pre, pre_bias, y, n = AT[:9]
    if not torch.cuda.is_available():
        for ok in (dict(), dict(y=None), dict(post=None, post_bias=None), dict(gate=None, R=1), dict(pre=None, pre_bias=None, n=None),
                   dict(M=0, R=4), dict(weights_dtype=2), dict(b=None, post=None, post_bias=None, gate=None, y=None, R=1), dict(b=x),
                   dict(x=x + 2), dict(N=16384), dict(R=6)):
            assert call(**ok) in PAST_THE_CHECKS, ok
    for bad in (dict(x=None), dict(b=None), dict(post=None), dict(pre=None), dict(n=None), dict(pre=None, pre_bias=None),
                dict(y=None, n=None, pre=None, pre_bias=None), dict(gate=None), dict(R=4), dict(R=0), dict(R=12), dict(N=0), dict(N=16385),
                dict(M=-1), dict(M=1 << 31), dict(dtype=3), dict(weights_dtype=1), dict(x=x + 1), dict(post=post + 2), dict(y=x), dict(y=b),
                dict(n=y), dict(n=y + 2), dict(y=gate), dict(n=pre), dict(n=pre_bias)):
        assert call(**bad) == BAD, bad
    assert L.block_norm(None, None) == BAD


def test_block_norm_backward_refusals(L):
    names = [f[0] for f in NormBackwardCall._fields_]
    at = dict(zip(names, AT))
    need, ws = L.block_norm_backward_workspace_size(6, 64, 2, 2), AT[20]
    call = lambda to=ws, size=need, **kw: held(L.block_norm_backward, norm_call(NormBackwardCall, **kw), to, size, None)  # noqa: E731
    gone = dict(b=None, post=None, post_bias=None, gate=None, db=None, dgate=None, dpost=None, dpost_bias=None, R=1)
    if not torch.cuda.is_available():
        for ok in (dict(), dict(dy=None), dict(dx=None), dict(db=None), dict(dgate=None), dict(dpost=None), dict(dpre=None), gone,
                   dict(pre=None, pre_bias=None, dn=None, y=None, dpre=None, dpre_bias=None)):
            assert call(**ok) in PAST_THE_CHECKS, ok
    for bad in (dict(dn=None), dict(y=None), dict(b=None), dict(post=None), dict(gate=None), dict(pre=None), dict(R=4), dict(N=0),
                dict(dtype=3), dict(weights_dtype=1), dict(dx=at["dy"]), dict(db=at["b"]), dict(dgate=at["dpost"]), dict(dpre=at["gate"]),
                dict(dx=at["db"]), dict(dy=None, dn=None, pre=None, pre_bias=None, y=None, dpre=None, dpre_bias=None),
                dict(dgate=at["dgate"] + 2), dict(dx=at["dx"] + 1)):
        assert call(**bad) == BAD, bad
    for to in (*(at[n] for n in names[:16]), ws + 16, None, at["dy"] - need + 256):
        assert call(to=to) == BAD, to
    assert call(size=need - 1) == BAD and L.block_norm_backward(None, ws, need, None) == BAD


def test_block_norm_backward_workspace(L):
    size = L.block_norm_backward_workspace_size
    assert size(0, 64, 1, 0) == 0
    for m, n, r in ((1, 1, 1), (7, 100, 7), (4096, 4096, 1), (1000, 64, 500), (300, 16384, 3)):
        assert size(m, n, r, 2) >= 4 * n * 4, (m, n, r)
    for bad in ((5, 64, 2, 0), (-1, 64, 1, 0), (5, 0, 1, 0), (5, 64, 0, 0), (5, 64, 1, 3), (5, 16385, 1, 0), (2, 64, 4, 0)):
        assert size(*bad) == 0, bad


def test_compiled_calls_refuse(L):
    calls = bw._calls()
    for f in (calls.linear, calls.layer, calls.block, calls.block_backward):
        with pytest.raises(TypeError):
            f()
    x = torch.zeros((2, 128))
    with pytest.raises(TypeError):
        bw.block_norm(x, pre=torch.zeros(128))  # not on the GPU
    with pytest.raises(TypeError):
        bw.block_norm([1.0], pre=x)
    with pytest.raises(ValueError):
        bw.block_norm(x, pre=x, kind="both")
    with pytest.raises(TypeError):
        bw.block_norm_backward(x, x, dn=x, pre=torch.zeros(128))
    with pytest.raises(ValueError):
        bw.block_norm_backward(None, x)


@pytest.mark.parametrize("name", [None, "relu", "gelu", "gelu_tanh", "silu"])
def test_activations_of_the_reference(name):
    z = torch.linspace(-9, 9, 2001, dtype=torch.float64)
    f = torch.nn.functional
    want = {None: lambda v: v, "relu": f.relu, "gelu": f.gelu, "gelu_tanh": lambda v: f.gelu(v, approximate="tanh"), "silu": f.silu}[name]
    assert torch.allclose(act64(name, z), want(z), rtol=1e-12, atol=1e-15)
    assert act64(name, torch.tensor([-math.inf], dtype=torch.float64)).item() == (0.0 if name else -math.inf)


def test_norms_of_the_reference():
    v = torch.randn((5, 33), dtype=torch.float64)
    assert torch.allclose(hat64(v, "layer", 1e-5), torch.nn.functional.layer_norm(v, (33,), eps=1e-5), rtol=1e-12)
    h = hat64(v, "rms", 0.0)
    assert torch.allclose((h * h).mean(1), torch.ones(5, dtype=torch.float64)) and torch.allclose(h / v, (h / v)[:, :1].expand(5, 33))
