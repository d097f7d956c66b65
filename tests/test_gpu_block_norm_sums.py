"""GPU: the norms and their parameter gradients as the C entry points give them, each asked for by itself.

A bias's gradient needs no bias (it is a sum of dn or of du): its bits are the same with a bias of zeros and with none.  Against
64 bits: sums over M rows in any order round at most M - 1 times (2^-24 each, f32), and a row's terms are within 64 2^-24 of what
their formula adds: a thread sums at most 32 terms of a row in f32, threads are added in f64, and the formula's own operations
are fewer than sixteen.
"""

import ctypes
import itertools

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import CODES, NormBackwardCall, NormCall, hat64
from gpu_util import note
from q4_util import DTYPES, gen

pytestmark = pytest.mark.gpu
EPS = 1e-6
SUMS = ("dgate", "dpost", "dpost_bias", "dpre", "dpre_bias")


def backward(m, n, r, dtype, scale, ins, asked, kind="rms"):
    """The C call with the tensors `ins` and the outputs `asked`; whatever it does not write stays NaN."""
    L = bw.lib()
    nan = lambda *s, t=torch.float32: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    outs = {k: nan(m, n, t=DTYPES[dtype]) if k in ("dx", "db") else nan(r, n) if k == "dgate" else nan(n) for k in asked}
    need = L.block_norm_backward_workspace_size(m, n, r, CODES[dtype])
    ws = torch.full((need // 4 + 64,), float("nan"), device="cuda")
    at = -ws.data_ptr() % 256 // 4
    call = NormBackwardCall(**{k: v.data_ptr() for k, v in (*ins.items(), *outs.items()) if v is not None}, eps=EPS, M=m, N=n, R=r,
                            scale=scale, layer=kind == "layer", dtype=CODES[dtype], weights_dtype=CODES[dtype])
    st = L.block_norm_backward(ctypes.addressof(call), ws.data_ptr() + 4 * at, need, None)
    torch.cuda.synchronize()
    assert st == 0, st
    return outs


def rows(m, n, dtype, gates, post=True, pre=True, seed=1):
    t, g = DTYPES[dtype], gen(seed)
    rand = lambda *s, about=0.0, width=1.0: (about + width * torch.randn(s, generator=g)).to(t).cuda()  # noqa: E731
    ins = dict(b=rand(m, n), y=rand(m, n, width=2.0), dy=rand(m, n, width=0.5), dn=rand(m, n, width=0.5),
               gate=rand(gates, n, about=0.5, width=0.3), post=rand(n, about=1.0, width=0.1), pre=rand(n, about=1.0, width=0.1))
    for name, on in (("post", post), ("pre", pre)):
        if not on:
            ins[name] = None
    if not pre:
        ins["y"] = ins["dn"] = None
    return ins


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,gates", [(1, 5, 1), (40, 264, 1), (600, 264, 3), (33, 1111, 33), (12, 4096, 2), (6, 9001, 1)])
def test_bias_gradients_without_biases(m, n, gates, dtype):
    ins, scale = rows(m, n, dtype, gates), 0.7
    zeros = torch.zeros(n, dtype=DTYPES[dtype], device="cuda")
    note(f"[block_norm_backward] bias gradients without biases M={m} N={n} gates={gates} {dtype}")
    want = backward(m, n, gates, dtype, scale, dict(ins, post_bias=zeros, pre_bias=zeros), ("dx", "db", *SUMS))
    dn, gate = ins["dn"].double(), ins["gate"].double().repeat_interleave(m // gates, 0)
    hat, y = hat64(ins["y"].double(), "rms", EPS), ins["y"].double()
    rstd = 1 / ((y * y).mean(1, keepdim=True) + EPS).sqrt()
    g = dn * ins["pre"].double()
    mean = lambda v: v.mean(1, keepdim=True)  # noqa: E731
    du = scale * gate * (ins["dy"].double() + (g - hat * mean(g * hat)) * rstd)
    size = (scale * gate).abs() * (ins["dy"].double().abs() + (g.abs() + hat.abs() * mean((g * hat).abs())) * rstd)
    for name, terms, sizes in (("dpre_bias", dn, dn.abs()), ("dpost_bias", du, size)):
        err, tol = (want[name].double() - terms.sum(0)).abs(), (m + 64) * 2.0 ** -24 * sizes.sum(0)
        note(f"  {name} worst err/tol {float((err / tol).max()):.3g}")
        assert (err <= tol).all(), name
    for asked in (SUMS, ("dpre_bias",), ("dpost_bias",), ("dpre", "dpre_bias"), ("dx", "db", "dpost_bias")):
        got = backward(m, n, gates, dtype, scale, ins, asked)
        for name in asked:
            if "bias" in name:
                assert torch.equal(got[name], want[name]), (asked, name)
            assert not torch.isnan(got[name]).any(), (asked, name)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True)])
def test_any_selection_of_outputs(post, pre, kind):
    """An output's bits do not depend on which others are asked for (rms: with a bias's gradient among them, or without)."""
    m, n, gates = 26, 520, 2
    ins = rows(m, n, "bf16", gates, post, pre)
    names = [k for k in ("dx", "db", *SUMS) if (post or "post" not in k) and (pre or "pre" not in k)]
    note(f"[block_norm_backward] selections post={post} pre={pre} {kind}")
    biased = lambda asked: kind == "layer" or any("bias" in k for k in asked)  # noqa: E731
    want = {True: backward(m, n, gates, "bf16", 0.5, ins, names, kind),
            False: backward(m, n, gates, "bf16", 0.5, ins, [k for k in names if "bias" not in k], kind)}
    assert not any(torch.isnan(v).any() for v in want[True].values())
    for asked in itertools.chain(*(itertools.combinations(names, i) for i in (1, 2))):
        for name, v in backward(m, n, gates, "bf16", 0.5, ins, asked, kind).items():
            assert torch.equal(v, want[biased(asked)][name]), (asked, name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(1, 264), (5000, 100), (3001, 1111), (1300, 4096)])
def test_sums_over_rows_round_as_often_as_they_are_added(m, n, dtype):
    """The sum of dn: a workgroup adds its rows (M over their number, rounded up), a second kernel every 64th part and then
    64 sums in pairs: so many roundings of 2^-24, and no more, of what is added."""
    ins = rows(m, n, dtype, 1)
    ins["dn"] = (ins["dn"].float().abs() + 0.25).to(DTYPES[dtype])
    need = bw.lib().block_norm_backward_workspace_size(m, n, 1, CODES[dtype])
    parts = need // (4 * 5 * n) if m > 1 else 1  # four sums' parts and the gate's
    assert need == (5 if m > 1 else 4) * 4 * n * parts
    note(f"[block_norm_backward] {parts} parts M={m} N={n} {dtype}")
    got = backward(m, n, 1, dtype, 1.0, ins, ("dpre_bias",))["dpre_bias"].double()
    want = ins["dn"].double().sum(0)
    err, tol = (got - want).abs() / want, 2.0 ** -24 * (-(-m // parts) + -(-parts // 64) + 6)
    note(f"  worst err/tol {float(err.max() / tol):.3g}")
    assert (err <= tol).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_sum_need_not_be_kept(dtype, kind):
    """Without y the normed rows are the same; the sum's rounding to its type is part of them."""
    m, n, t = 37, 1000, DTYPES[dtype]
    ins = rows(m, n, dtype, 1)
    x = ins["y"]
    y, want = bw.block_norm(x, b=ins["b"], post=ins["post"], gate=ins["gate"], scale=0.7, pre=ins["pre"], kind=kind)
    got = torch.full((m, n), float("nan"), dtype=t, device="cuda")
    call = NormCall(x=x.data_ptr(), b=ins["b"].data_ptr(), post=ins["post"].data_ptr(), gate=ins["gate"].data_ptr(),
                    pre=ins["pre"].data_ptr(), n=got.data_ptr(), eps=EPS, M=m, N=n, R=1, scale=0.7, layer=kind == "layer",
                    dtype=CODES[dtype], weights_dtype=CODES[dtype])
    note(f"[block_norm] without the sum {kind} {dtype}")
    assert bw.lib().block_norm(ctypes.addressof(call), None) == 0
    torch.cuda.synchronize()
    assert torch.equal(got, want)
