"""Outputs of the 4-bit products that are infinite or NaN, or whose f32 sums overflow on the way to a finite result.

With up to 32 rows, and in the experts' products of few slots, codes are decoded to 16 + code and the rest is taken
off each group's sum; an output that does not come out finite is formed again term by term.  Here such outputs meet
every group size, zero points, K inside a unit, every type, and the last column of the last block.

Expected: the sum of x (code - zero) scale in f64, where an infinity times a weight of 0 is NaN.  Finite results are one
term of magnitude 2^120 and others below 2^-24 of it: half a step of the result's type, and f32's.
"""

import math

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import DTYPES, cuda, dequant64, gen, weight
from test_gpu_q4 import run

pytestmark = pytest.mark.gpu
INF = math.inf


def same(got, want, rel):
    got, want = got.double().cpu(), want.cpu()
    fin = torch.isfinite(want)
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    assert torch.isfinite(got[fin]).all() and ((got - want)[fin].abs() <= rel * want[fin].abs() + 2.0 ** -24).all()


def by_terms(x, wd):
    """x W^T in f64, term by term: a product's own order of operations may turn an infinity into NaN."""
    return (x.double()[:, None, :] * wd[None]).sum(-1)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 40, 512), (5, 33, 640), (17, 300, 256), (32, 17, 1152), (8, 4100, 128)])
def test_infinities_and_nan_in_few_rows(m, n, k, group, dtype):
    w = weight(1, (), n, k, group, True)
    wd = dequant64(*w)
    x = torch.randn((m, k), generator=gen(2)).to(DTYPES[dtype])
    at = torch.randint(0, k, (m,), generator=gen(3))
    kind = torch.arange(m) % 4
    for i in range(m):
        if kind[i] < 3:
            x[i, at[i]] = (INF, -INF, math.nan)[int(kind[i])]
    if m > 4:
        x[4, (at[4] + 1) % k] = -INF  # a second infinity
    note(f"[q4_gemm] not finite M={m} N={n} K={k} G={group} {dtype}")
    y = run(x.cuda(), w, dtype)
    clean = torch.where(x.isfinite(), x, 0).double() @ wd.T
    want = torch.where((~x.isfinite()).any(1)[:, None], by_terms(x, wd), clean)
    y = y.cpu()
    bad = ~torch.isfinite(want)
    assert torch.equal(y.isnan(), want.isnan()) and torch.equal(y[want.isinf()].double(), want[want.isinf()])
    assert torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group,k", [(32, 160), (64, 320), (128, 1024)])
@pytest.mark.parametrize("m", [1, 9, 32, 100])
def test_sums_that_overflow_on_the_way_to_a_finite_result(m, group, k, dtype):
    """x of 2^125: (16 + code) x does not fit f32, (code - zero) scale x does."""
    n = 50
    w = weight(4, (), n, k, group, True, scale=2.0 ** -9)
    x = torch.randn((m, k), generator=gen(5)).to(DTYPES[dtype])
    x[torch.arange(m), torch.randint(0, k, (m,), generator=gen(6))] = 2.0 ** 125
    note(f"[q4_gemm] large values M={m} G={group} {dtype}")
    y = run(x.cuda(), w, dtype)
    want = x.double() @ dequant64(*w).T
    # where the large one meets a weight of 0, the others' sum may be lost beside it
    large = want.abs() > 2.0 ** 100
    eps = torch.finfo(DTYPES[dtype]).eps
    same(torch.where(large, y.cpu().double(), 0), torch.where(large, want, 0), eps / 2 + 2.0 ** -20)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,e,k", [(1, 8, 4), (3, 8, 4), (40, 64, 1), (30, 16, 4), (300, 4, 2)])
def test_experts_rows_that_are_not_finite_stay_by_themselves(t, e, k, dtype):
    d, f = 128, 160
    w = [weight(7, (e,), f, d, 32, True), weight(8, (e,), f, d, 32, True), weight(9, (e,), d, f, 32, True)]
    x = torch.randn((t, d), generator=gen(10)).to(DTYPES[dtype])
    x[0, 5] = math.nan
    if t > 2:
        x[2, 7] = INF
    idx = torch.stack([torch.randperm(e, generator=gen(20 + i))[:k] for i in range(t)]).int()
    wts = torch.rand((t, k), generator=gen(11)) + 0.1
    handles = [bw.q4_upload(*(cuda(v) for v in m)) for m in w]
    note(f"[q4_moe] not finite T={t} E={e} k={k} {dtype}")
    y = bw.q4_moe(x.cuda(), idx.cuda(), wts.cuda(), *handles)
    assert y[0].isnan().all()
    if t > 2:
        assert not torch.isfinite(y[2]).any()
    rest = [i for i in range(t) if i not in (0, 2)]
    if rest:
        clean = torch.where(x.isfinite(), x, 0)
        assert torch.equal(y[rest], bw.q4_moe(clean.cuda(), idx.cuda(), wts.cuda(), *handles)[rest])
