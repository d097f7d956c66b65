"""GPU parity of the 4-bit weight product, its packing and its decode with 64-bit references.

Tolerances.  q4_dequant is exact in f32 ((code - zero) has at most 5 bits beside the
f16 scale's 11).  q4_gemm's products are exact; its f32 sums run over terms of magnitude
up to (16 + code) scale |x| and (16 + zero) scale |x|, so with B = sum |x| scale each is
bounded by 31 B, a group of G terms in up to three parts, then the groups and eight waves:
at most (3 G + K/G + 16) roundings of 2^-24 on partial sums below 62 B.  The result is rounded
once to the output's type: eps/2 of its value.  In the 2-norm the f32 sums' part is far
smaller (roundings of either sign): 2^-20 of the result's norm.  More than 64 rows of 16-bit
or f32 x may take the prompt kernel: weights of a bfloat16 product are then rounded to
f16 (2^-12 of each term, so at most 2^-12 sum |x w|, and 2^-11 of the norm).
"""

import numpy as np
import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import DTYPES, cuda, dequant64, gen, weight

pytestmark = pytest.mark.gpu


def check(y, x, w, dtype, what):
    codes, scales, zeros = w
    wd = dequant64(*w).cuda()
    k = wd.shape[1]
    group = k // scales.shape[1]
    x64 = x.double()
    want = x64 @ wd.T.contiguous()
    s64 = scales.double().cuda().repeat_interleave(group, -1).abs()
    b = x64.abs() @ s64.T.contiguous()
    eps = torch.finfo(DTYPES[dtype]).eps
    tol = eps / 2 * want.abs() + (3 * group + k // group + 16) * 2.0 ** -24 * 62 * b
    norm = eps / 2 + 2.0 ** -20
    if dtype == "bf16" and x.shape[0] > 64:
        tol = tol + 2.0 ** -12 * (x64.abs() @ wd.abs().T.contiguous())
        norm += 2.0 ** -11
    if dtype == "f16":
        tol = tol + 2.0 ** -25  # subnormal results
    err = (y.double() - want).abs()
    rel = float((err.norm() / want.norm()).item()) if want.norm() else float(err.norm())
    note(f"  {what}: rel {rel:.3g} (allowed {norm:.3g}), worst err/tol {float((err / tol.clamp_min(1e-300)).max()):.3g}")
    assert torch.isfinite(y).all(), what
    assert (err <= tol).all(), what
    assert rel <= norm, what


def run(x, w, dtype):
    """q4_gemm into a poisoned buffer with a guarded tail."""
    h = bw.q4_upload(*(cuda(t) for t in w))
    m, n = x.shape[0], h.N
    base = torch.full((m * n + 64,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    y = base[: m * n].view(m, n)
    assert bw.q4_gemm(h, x, y) is y
    torch.cuda.synchronize()
    assert torch.isnan(base[m * n:]).all(), "write past the end of y"
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("lead,n,k", [((), 1, 128), ((), 40, 384), ((3,), 17, 256), ((), 1000, 640)])
def test_dequant_is_exact(lead, n, k, zeros, group):
    w = weight(1, lead, n, k, group, zeros)
    note(f"[q4_dequant] lead={lead} N={n} K={k} G={group} zeros={zeros}")
    h = bw.q4_upload(*(cuda(t) for t in w))
    got = bw.q4_dequant(h).cpu()
    assert got.shape == (*lead, n, k)
    assert torch.equal(got.double(), dequant64(*w))


def test_dequant_of_odd_groups_and_extreme_scales():
    """K that ends inside a unit of 128, and scales that are negative, subnormal, largest and zero."""
    codes, scales, zeros = weight(2, (), 33, 4000, 32, True)
    scales[0, :6] = torch.tensor([-0.5, 2.0 ** -24, -(2.0 ** -20), 65504.0, -65504.0, 0.0]).half()
    note("[q4_dequant] extreme scales")
    h = bw.q4_upload(codes.cuda(), scales.cuda(), zeros.cuda())
    assert torch.equal(bw.q4_dequant(h).cpu().double(), dequant64(codes, scales, zeros))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", [1, 2, 15, 16, 17, 33, 64, 65, 130])
@pytest.mark.parametrize("n,k,group,zeros", [(64, 256, 128, False), (100, 4000, 32, True), (1500, 1216, 64, True),
                                             (9, 32, 32, False)])
def test_gemm(m, n, k, group, zeros, dtype):
    w = weight(3, (), n, k, group, zeros)
    x = torch.randn((m, k), generator=gen(4)).to(DTYPES[dtype]).cuda()
    note(f"[q4_gemm] M={m} N={n} K={k} G={group} zeros={zeros} {dtype}")
    y = run(x, w, dtype)
    check(y, x, w, dtype, f"M={m}")
    again = run(x, w, dtype)
    assert torch.equal(y.view(torch.uint8), again.view(torch.uint8)), "not deterministic"


@pytest.mark.parametrize("dtype,m,n,k,group", [("bf16", 1, 9000, 8192, 128), ("f16", 8, 20000, 1024, 32),
                                               ("f32", 40, 5003, 4000, 32), ("bf16", 300, 4096, 1024, 128),
                                               ("f16", 257, 1000, 2048, 64), ("f32", 129, 2050, 1024, 128),
                                               ("bf16", 1000, 511, 4096, 32)])
def test_gemm_larger(dtype, m, n, k, group):
    w = weight(5, (), n, k, group, True)
    x = torch.randn((m, k), generator=gen(6)).to(DTYPES[dtype]).cuda()
    note(f"[q4_gemm] M={m} N={n} K={k} G={group} {dtype}")
    check(run(x, w, dtype), x, w, dtype, f"M={m} N={n}")


@pytest.mark.parametrize("m", [5, 200])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gemm_rows_of_very_different_size(dtype, m):
    """Rows from 1e-30 to 1e30 and rows of zeros keep their own precision; a row's outliers do not drown it."""
    n, k = 96, 1024
    w = weight(7, (), n, k, 128, False)
    x = torch.randn((m, k), generator=gen(8))
    x = x * torch.logspace(-30, 30, m)[:, None]
    x[m // 2] = 0
    x[1, 3] *= 1e4
    x = x.to(DTYPES[dtype]).cuda()
    note(f"[q4_gemm] rows of very different size M={m} {dtype}")
    y = run(x, w, dtype)
    assert (y[m // 2] == 0).all()
    want = x.double() @ dequant64(*w).cuda().T.contiguous()
    live = [i for i in range(m) if i != m // 2]
    rel = ((y.double() - want).norm(dim=1) / want.norm(dim=1))[live]
    # as in check(): rounding of the result, f32 sums, and the prompt kernel's weights
    assert float(rel.max()) <= torch.finfo(DTYPES[dtype]).eps / 2 + 2.0 ** -20 + (2.0 ** -11 if m > 64 and dtype == "bf16" else 0)


@pytest.mark.parametrize("m", [3, 100])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gemm_infinities_and_nan_stay_in_their_rows(dtype, m):
    n, k = 48, 256
    codes, scales, _ = weight(9, (), n, k, 64, False)
    codes[:, 4] = 0x9F  # elements 8 and 9: codes 15 and 9, both above the zero point 8
    x = torch.randn((m, k), generator=gen(10)).to(DTYPES[dtype])
    x[0, 8] = float("inf")
    x[1, 9] = float("nan")
    note(f"[q4_gemm] Inf and NaN rows M={m} {dtype}")
    y = run(x.cuda(), (codes, scales, None), dtype).cpu()
    assert (y[0] == float("inf")).all()
    assert torch.isnan(y[1]).all()
    assert torch.isfinite(y[2:]).all()


@pytest.mark.parametrize("m", [2, 80])
def test_gemm_extreme_scales(m):
    """Scales at both ends of f16 in one weight; K ends inside a unit."""
    n, k, group = 64, 160, 32
    codes, scales, zeros = weight(11, (), n, k, group, True)
    scales[:20] = (scales[:20].float() * 2.0 ** 18).clamp(max=60000.0).half()
    scales[20:40] = (scales[20:40].float() * 2.0 ** -12).half()
    w = (codes, scales, zeros)
    x = torch.randn((m, k), generator=gen(12)).bfloat16().cuda()
    note(f"[q4_gemm] extreme scales M={m}")
    y = run(x, w, "bf16")
    want = x.double() @ dequant64(*w).cuda().T.contiguous()
    err = (y.double() - want).norm(dim=0) / want.norm(dim=0)
    assert float(err.max()) <= 2.0 ** -8 + 2.0 ** -20 + 2.0 ** -11


def test_gemm_on_a_row_slice_and_another_stream():
    n, k = 128, 512
    w = weight(13, (), n, k, 128, False)
    h = bw.q4_upload(*(cuda(t) for t in w))
    x = torch.randn((40, k), generator=gen(14)).bfloat16().cuda()
    note("[q4_gemm] slice of rows, side stream")
    whole = bw.q4_gemm(h, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    part = bw.q4_gemm(h, x[7:12], stream=side)
    side.synchronize()
    # same rows, same numbers: a row's sums do not depend on the rows beside it
    assert torch.equal(part, whole[7:12])
    assert bw.q4_gemm(h, x[:0]).shape == (0, n)


@pytest.mark.parametrize("m", [1, 24, 200])
def test_gemm_in_a_graph(m):
    n, k = 1024, 1024
    w = weight(15, (), n, k, 64, True)
    h = bw.q4_upload(*(cuda(t) for t in w))
    x = torch.randn((m, k), generator=gen(16)).bfloat16().cuda()
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    note(f"[q4_gemm] graph M={m}")
    bw.q4_gemm(h, x, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bw.q4_gemm(h, x, y)
    for rep in range(4):
        x.copy_(torch.randn((m, k), generator=gen(17 + rep)).bfloat16())
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bw.q4_gemm(h, x)), rep
        torch.cuda.synchronize()
