"""GPU: q4_linear's activations by themselves, at products that are exact.

A weight's row has one 1 and else zeros, so that z is x's first element, exactly, on every path (16 + code times x needs five bits
more than x has, and x's rows have one value other than 0).  What is left is the activation's own error and one rounding.
Bounds, relative to the result, in steps of 2^-24, with t the exponent (v for silu, 2 sqrt(2/pi) (v + 0.044715 v^3) for the form with
tanh, v^2 / 2 for gelu): t has at most six roundings (two constants', three products' and a sum's, the one with log2(e) among
them; erfc's argument two of v, four of v^2 / 2), which e^t multiplies by |t|; exp2, the reciprocal, erfc (sixteen) and the
sums 32 more.  The polynomial for 16-bit results is within 2^-16 by itself: 2^-24 (6 |t| + 32) + 2^-16 for 16 bits (an f16 half step is
2^-11, a bf16 one 2^-8), 2^-24 (6 |t| + 32) for f32.  What is below f32's normal range may be flushed to 0: a result (2^-126), or
the factor 1 / (1 + e^t), which is 0 from e^t = 2^126 or 2^128 on, where v times it is below |v| 2^-126.
"""

import math

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import half_step, least
from gpu_util import note
from q4_util import DTYPES

pytestmark = pytest.mark.gpu


def act64(act, z):
    """The activations in f64 without a difference that cancels: v s(t), v Phi(v) by erfc."""
    if act == "relu":
        return z.clamp(min=0)
    out = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) if act == "gelu" else z / (1.0 + torch.exp(-exponent(act, z) * z.sign()))
    return torch.where(z == -math.inf, 0.0, out)


def exponent(act, z):
    if act == "gelu":
        return z * z / 2
    return 2 * math.sqrt(2 / math.pi) * (z.abs() + 0.044715 * z.abs() ** 3) if act == "gelu_tanh" else z.abs()


def one(n, k):
    """W[n][0] = 1, the rest 0."""
    codes = torch.full((n, k // 2), 0x88, dtype=torch.uint8)
    codes[:, 0] = 0x89
    return bw.q4_upload(codes.cuda(), torch.ones((n, k // 128)).half().cuda())


def values(count, t):
    """Dense where activations bend, and wide beyond."""
    near = torch.linspace(-7, 7, count - count // 4, dtype=torch.float64)
    far = torch.linspace(-13, -5, count // 4, dtype=torch.float64)
    v = torch.cat((near, far)).half()  # (f32's too: 22 bits go through its two f16 parts)
    return v.to(t)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 128), (9, 40, 128), (25, 17, 256), (300, 24, 128), (300, 264, 8192), (2048, 264, 1024), (2050, 5, 256)])
def test_activation(m, n, k, act, dtype):
    t = DTYPES[dtype]
    h, rounds = one(n, k), -(-1600 // m)
    note(f"[q4_linear] activation {act} M={m} N={n} K={k} {dtype}")
    all_v, worst = values(rounds * m, t), 0.0
    for i in range(rounds if m < 100 else 1):
        x = torch.zeros((m, k), dtype=t)
        x[:, 0] = all_v[i::rounds][:m] if m < 100 else all_v[:m]
        y = bw.q4_linear(h, x.cuda(), activation=act).cpu().double()
        z = x[:, :1].double()
        want = act64(act, z).expand(m, n)
        own = 0.0 if act == "relu" else 2.0 ** -24 * (6 * exponent(act, z) + 32) + (0.0 if dtype == "f32" else 2.0 ** -16)
        tol = want.abs() * (own + half_step(dtype) * 1.01) + least(dtype) + 2.0 ** -126 * (1 + z.abs())
        err = (y - want).abs()
        worst = max(worst, float((err / tol).max()))
        assert (err <= tol).all(), (i, float(z[(err > tol).any(1)][0]))
    note(f"  worst err/tol {worst:.3g}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("m", [9, 300, 2048])
def test_limits_in_16_bits(m, act, dtype):
    """Infinite, huge and tiny products: what the formula tends to, and no NaN but a NaN's."""
    t = DTYPES[dtype]
    big = torch.finfo(t).max
    v = torch.tensor([-math.inf, -big, -1000.0, -30.0, -0.0, 0.0, 2.0 ** -20, 30.0, big], dtype=t)
    x = torch.zeros((m, 128), dtype=t)
    x[:, 0] = v.repeat(-(-m // 9))[:m]
    x[1::9, 0] = math.inf
    note(f"[q4_linear] limits {act} M={m} {dtype}")
    plain = bw.q4_gemm(one(16, 128), x.cuda()).double()
    y = bw.q4_linear(one(16, 128), x.cuda(), activation=act).cpu().double()
    want = act64(act, plain).cpu()  # (beside an infinity a prompt's row may be NaN: the product's own)
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and torch.equal(torch.isinf(y), torch.isinf(want))
    fin = torch.isfinite(want)
    own = 2.0 ** -24 * (6 * exponent(act, plain.cpu()).clamp(max=400) + 32) + 2.0 ** -16 + half_step(dtype) * 1.01
    assert ((y - want).abs() <= want.abs() * own + least(dtype) + 2.0 ** -126)[fin].all()
