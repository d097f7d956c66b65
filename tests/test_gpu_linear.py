"""GPU parity of the 4-bit product with its epilogue, y = act(x W^T + bias) + residual, with a 64-bit reference.

Tolerances, element by element.  The product as q4_gemm's: at most (3 G + K/G + 32) roundings of 2^-24 on partial sums below
62 B, B = sum |x| scale.  The activations' slopes are below 1.13; their own arithmetic, the bias and the residual are some
sixteen roundings of 2^-24 of 1 + |z| + |bias| + |residual| (an error of |t| 2^-23 in e^-t counts t s (1 - s) |v| 2^-23 in v s(t), below
2^-22; the argument of erfc, v / sqrt 2 rounded, v^2 2^-24 of v Phi(v), below 2^-24).  The result is rounded once: half a step of its type.
"""

import math
import warnings

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import act64, half_step, least
from gpu_util import note
from q4_util import DTYPES, cuda, dequant64, gen, weight

pytestmark = pytest.mark.gpu
ACTS = [None, "relu", "gelu", "gelu_tanh", "silu"]


def inputs(m, n, k, dtype, bias, residual, seed=1):
    t = DTYPES[dtype]
    x = torch.randn((m, k), generator=gen(seed)).to(t)
    b = None if bias is None else (0.5 * torch.randn(n, generator=gen(seed + 1))).to(DTYPES[bias])
    r = (2 * torch.randn((m, n), generator=gen(seed + 2))).to(t) if residual else None
    return x.cuda(), cuda(b), cuda(r)


def reference(x, w, bias, act, residual):
    codes, scales, zeros = w
    wd, x64 = dequant64(*w).cuda(), x.double()
    k, group = wd.shape[1], wd.shape[1] // scales.shape[1]
    z = x64 @ wd.T.contiguous()
    if bias is not None:
        z = z + bias.double()
    want = act64(act, z)
    if residual is not None:
        want = want + residual.double()
    b = x64.abs() @ scales.double().cuda().abs().repeat_interleave(group, -1).T.contiguous()
    size = 1 + z.abs() + (0 if bias is None else bias.double().abs()) + (0 if residual is None else residual.double().abs())
    return want, 1.13 * (3 * group + k // group + 32) * 2.0 ** -24 * 62 * b + 16 * 2.0 ** -24 * size


def check(m, n, k, group, zeros, dtype, act, bias, residual, inplace=False):
    w = weight(3, (), n, k, group, zeros)
    x, b, r = inputs(m, n, k, dtype, bias, residual)
    want, tol = reference(x, w, b, act, r)
    tol = tol + half_step(dtype) * want.abs() + least(dtype)
    h = bw.q4_upload(*(cuda(t) for t in w))
    note(f"[q4_linear] M={m} N={n} K={k} G={group} zeros={zeros} {dtype} act={act} bias={bias} residual={residual} in place={inplace}")
    base = torch.full((m * n + 64,), float("nan"), dtype=DTYPES[dtype], device="cuda")
    y = base[: m * n].view(m, n)
    if inplace:
        y.copy_(r)
        r = y
    assert bw.q4_linear(h, x, bias=b, activation=act, residual=r, y=y) is y
    torch.cuda.synchronize()
    assert torch.isnan(base[m * n:]).all(), "write past the end of y"
    err = (y.double() - want).abs()
    note(f"  worst err/tol {float((err / tol).max()):.3g}")
    assert (err <= tol).all()
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k,group,zeros", [(1, 100, 256, 128, False), (7, 1000, 1216, 64, True), (20, 4100, 512, 32, True),
                                               (33, 520, 640, 32, False), (130, 515, 4096, 128, True)])
def test_linear(m, n, k, group, zeros, act, dtype):
    check(m, n, k, group, zeros, dtype, act, "f32" if m % 2 else dtype, m != 7)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bias,residual", [(None, False), ("own", False), (None, True), ("own", True)])
@pytest.mark.parametrize("m,n,k,group", [(2, 17, 128, 64), (40, 260, 384, 128), (257, 1000, 2048, 64), (700, 1030, 512, 32)])
def test_parts_of_the_epilogue(m, n, k, group, bias, residual, dtype):
    check(m, n, k, group, True, dtype, "silu" if m == 40 else None, dtype if bias else None, residual)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,k,group", [(1, 9, 32, 32), (3, 511, 1024, 64), (200, 1111, 4096, 128), (1030, 2050, 256, 128)])
def test_in_place_of_the_residual(m, n, k, group, dtype):
    check(m, n, k, group, False, dtype, "gelu", "f32", True, inplace=True)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m", [1, 20, 100, 600])
def test_an_empty_epilogue_is_the_product(m, dtype):
    w = weight(5, (), 1040, 1024, 64, True)
    x = inputs(m, 1040, 1024, dtype, None, False)[0]
    h = bw.q4_upload(*(cuda(t) for t in w))
    note(f"[q4_linear] empty epilogue M={m} {dtype}")
    assert torch.equal(bw.q4_linear(h, x), bw.q4_gemm(h, x))


@pytest.mark.parametrize("act", ACTS)
def test_limits_of_the_activations(act):
    """Products from -1000 to 1000 and infinite ones: what the formula tends to, with no NaN of -inf * 0."""
    k = 128
    codes = torch.full((6, k // 2), 0x88, dtype=torch.uint8)
    codes[:, 0] = 0x89  # element 0 is 1, the rest 0
    h = bw.q4_upload(codes.cuda(), torch.ones((6, 1)).half().cuda())
    x = torch.zeros((9, k))
    x[:, 0] = torch.tensor([-math.inf, -1000.0, -100.0, -20.0, -1.0, 1.0, 20.0, 1000.0, math.inf])
    note(f"[q4_linear] limits {act}")
    y = bw.q4_linear(h, x.cuda(), activation=act).cpu().double()
    want = act64(act, x[:, :1].double()).expand(9, 6)
    assert torch.equal(torch.isinf(y), torch.isinf(want)) and not torch.isnan(y).any()
    fin = torch.isfinite(want)
    # f32's subnormals may be flushed; |v|^2 2^-23 of e^-t's argument
    assert ((y - want).abs()[fin] <= (2.0 ** -20 * want.abs() * 20 + 2.0 ** -126)[fin]).all()


def test_rows_with_nan_and_infinities_stay_apart():
    w = weight(7, (), 300, 512, 64, True)
    h = bw.q4_upload(*(cuda(t) for t in w))
    for m in (4, 150):
        x, b, r = inputs(m, 300, 512, "bf16", "bf16", True)
        clean = bw.q4_linear(h, x, bias=b, activation="silu", residual=r)
        x[1, 7] = float("nan")
        note(f"[q4_linear] NaN row M={m}")
        y = bw.q4_linear(h, x, bias=b, activation="silu", residual=r)
        rest = [i for i in range(m) if i != 1]
        assert torch.isnan(y[1]).all() and torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("m", [1, 24, 300])
def test_in_a_graph_and_on_another_stream(m):
    n, k = 4099, 1024
    h = bw.q4_upload(*(cuda(t) for t in weight(9, (), n, k, 128, False)))
    x, b, r = inputs(m, n, k, "bf16", "f32", True)
    y = torch.empty((m, n), dtype=x.dtype, device="cuda")
    note(f"[q4_linear] graph M={m}")
    bw.q4_linear(h, x, bias=b, activation="gelu", residual=r, y=y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bw.q4_linear(h, x, bias=b, activation="gelu", residual=r, y=y)
    for rep in range(4):
        x.copy_(torch.randn((m, k), generator=gen(20 + rep)))
        b.copy_(torch.randn(n, generator=gen(30 + rep)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, bw.q4_linear(h, x, bias=b, activation="gelu", residual=r)), rep
        torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bw.q4_linear(h, x, bias=b, activation="gelu", residual=r, stream=side)
    side.synchronize()
    assert torch.equal(got, y)


def test_refusals_and_empty_calls():
    h = bw.q4_upload(*(cuda(t) for t in weight(11, (), 64, 128, 64, True)))
    x, b, r = inputs(8, 64, 128, "bf16", "bf16", True)
    note("[q4_linear] refusals")
    assert bw.q4_linear(h, x[:0], bias=b, residual=r[:0]).shape == (0, 64)
    with pytest.raises(TypeError):
        bw.q4_linear(h, x, bias=b.half())
    with pytest.raises(ValueError):
        bw.q4_linear(h, x, bias=b[:63])
    with pytest.raises(TypeError):
        bw.q4_linear(h, x, residual=r.float())
    with pytest.raises(ValueError):
        bw.q4_linear(h, x, residual=r[:7])
    with pytest.raises(ValueError):
        bw.q4_linear(h, x, residual=torch.empty((64, 8), dtype=x.dtype, device="cuda").T)
    with pytest.raises(ValueError):
        bw.q4_linear(h, x, activation="tanh")
    with pytest.raises(bw.Tq2Error):
        bw.q4_linear(h, x, residual=x.view(-1)[:512].view(8, 64), y=x.view(-1)[8:520].view(8, 64))
    wide = torch.zeros(9 * 64, dtype=x.dtype, device="cuda")
    with pytest.raises(bw.Tq2Error):  # overlaps the residual in part
        bw.q4_linear(h, x, residual=wide[:512].view(8, 64), y=wide[64:].view(8, 64))
    stack = bw.q4_upload(*(cuda(t) for t in weight(12, (2,), 64, 128, 64, False)))
    with pytest.raises(ValueError):
        bw.q4_linear(stack, x)
    with pytest.warns(UserWarning, match="q4_linear forms no gradient"):
        bw.q4_linear(h, x, bias=b.float().requires_grad_())
    with warnings.catch_warnings(), torch.no_grad():
        warnings.simplefilter("error")
        bw.q4_linear(h, x, residual=r.clone().requires_grad_())
