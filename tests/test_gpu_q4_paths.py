"""Every way in which the 4-bit products and the experts' products are dealt out, their calls' streams and
far offsets, and the example that runs them together.

Sizes of q4_gemm here are ones that take blocks of 32 rows side by side, tiles of 64 and of 128 rows, and the
units of k in several shares, with odd columns and K that ends inside a unit.  Tolerances are test_gpu_q4's: f32 sums
in up to 16 shares more add 16 roundings, inside the 16 that its bound leaves for waves.  The experts' products:
test_gpu_moe's.
"""

import importlib.util
import os

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import DTYPES, cuda, dequant64, gen, weight
from test_gpu_moe import check_moe
from test_gpu_q4 import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(33, 1040, 2048), (96, 4096, 1024), (129, 2051, 4096), (256, 1000, 8192),
                                   (300, 4100, 1152), (1100, 2048, 512), (2050, 4096, 384)])
def test_gemm_deals(m, n, k, group, dtype):
    w = weight(31, (), n, k, group, True)
    x = torch.randn((m, k), generator=gen(32)).to(DTYPES[dtype]).cuda()
    note(f"[q4_gemm] M={m} N={n} K={k} G={group} {dtype}")
    y = run(x, w, dtype)
    check(y, x, w, dtype, f"M={m}")
    assert torch.equal(y.view(torch.uint8), run(x, w, dtype).view(torch.uint8)), "not deterministic"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [4000, 160])
def test_gemm_deals_odd_units(k, dtype):
    """K that is no multiple of 128: the last share's unit is part of one."""
    w = weight(33, (), 2050, k, 32, True)
    x = torch.randn((200, k), generator=gen(34)).to(DTYPES[dtype]).cuda()
    note(f"[q4_gemm] K={k} {dtype}")
    check(run(x, w, dtype), x, w, dtype, f"K={k}")


@pytest.mark.parametrize("m", [40, 150, 520])
def test_gemm_deals_infinities_stay_in_their_rows(m):
    codes, scales, _ = weight(35, (), 2048, 2048, 128, False)
    codes[:, 4] = 0x9F  # elements 8 and 9: codes 15 and 9, both above the zero point 8
    x = torch.randn((m, 2048), generator=gen(36)).bfloat16()
    x[0, 8], x[m - 1, 9] = float("inf"), float("nan")
    note(f"[q4_gemm] Inf and NaN rows M={m}")
    y = run(x.cuda(), (codes, scales, None), "bf16").cpu()
    assert (y[0] == float("inf")).all() and torch.isnan(y[m - 1]).all() and torch.isfinite(y[1: m - 1]).all()


@pytest.mark.parametrize("m", [1, 20, 64, 260, 1200])
def test_gemm_subnormal_activations_are_exact(m):
    """f16 rows with one subnormal value each: every output is a small multiple of 2^-15, without any rounding."""
    n, k = 1040, 1024
    codes, scales, zeros = weight(39, (), n, k, 64, True)
    scales = torch.full_like(scales, 512.0)
    x = torch.zeros((m, k))
    at = torch.arange(m) * 7 % k
    x[torch.arange(m), at] = (1 + torch.arange(m) % 5) * 2.0 ** -24
    note(f"[q4_gemm] subnormal x M={m}")
    y = run(x.half().cuda(), (codes, scales, zeros), "f16")
    want = x.double()[torch.arange(m), at][:, None] * dequant64(codes, scales, zeros).T[at]
    assert torch.equal(y.cpu().double(), want)


def test_gemm_rows_past_32_bits():
    """Rows whose byte offsets (x, and x as f16 planes) pass 2^32."""
    m, n, k = 66000, 64, 32768
    w = weight(37, (), n, k, 128, False)
    h = bw.q4_upload(*(cuda(t) for t in w))
    x = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=gen(38, "cuda"))
    note(f"[q4_gemm] M={m} N={n} K={k}")
    y = bw.q4_gemm(h, x)
    for rows in (slice(0, 40), slice(m - 40, m)):
        check(y[rows], x[rows], w, "bf16", f"rows {rows.start} on")
    full = bw.q4_gemm(h, x[m - 200:])
    assert torch.isfinite(full).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,e,k,d,f,group", [(50, 64, 8, 128, 512, 128), (70, 64, 8, 160, 512, 32), (300, 64, 8, 128, 512, 64),
                                             (40, 8, 4, 2176, 128, 128), (25, 16, 2, 2048, 64, 64), (25, 16, 2, 64, 2048, 64),
                                             (90, 3, 3, 96, 320, 32)])
def test_moe_deals(t, e, k, d, f, group, dtype):
    """Slots that workgroups find, tiles of 64 and blocks of 16 rows; rows longer than a wave's registers."""
    check_moe(t, e, k, d, f, group, True, dtype, "deals", seed=90)


@pytest.mark.parametrize("t,k,e", [(4, 8, 32), (33, 1, 8), (129, 4, 16)])
def test_moe_between_the_deals(t, k, e):
    """Just at and past 32 slots, and a full set of rows of one expert beside others that are empty."""
    idx = torch.randint(0, e, (t, k), generator=gen(91))
    idx[:, 0] = 1
    check_moe(t, e, k, 256, 128, 64, False, "bf16", "between", idx=idx, seed=92)


def test_moe_weights_past_32_bits():
    """Codes of the last expert lie more than 2^32 bytes in."""
    e, n, k = 130, 8192, 8192
    codes = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen(93, "cuda"))
    scales = torch.full((e, n, k // 128), 0.2 / k ** 0.5, dtype=torch.float16, device="cuda")
    note(f"[q4_moe] E={e} N=K={n}")
    w = bw.q4_upload(codes, scales)
    x = torch.randn((40, k), generator=gen(94)).cuda()
    last = dequant64(codes[-1].cpu(), scales[-1].cpu(), None).cuda()
    for t in (1, 40):  # by row, and by blocks of rows
        idx = torch.full((t, 1), e - 1, dtype=torch.int32, device="cuda")
        y = bw.q4_moe(x[:t].contiguous(), idx, torch.ones((t, 1), device="cuda"), w, w, w)
        g = x[:t].double() @ last.T.contiguous()
        want = (g * g / (1 + torch.exp(-g))) @ last.T.contiguous()
        assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -18


def test_route_more_tokens_than_one_launch():
    t, e = (1 << 25) + 3, 2
    logits = torch.empty((t, e), dtype=torch.bfloat16, device="cuda").normal_(generator=gen(95, "cuda"))
    note(f"[moe_route] T={t}")
    idx, w = bw.moe_route(logits, 1)
    assert torch.equal(idx[:, 0].bool(), logits[:, 1] > logits[:, 0])
    assert float(w.min()) >= 0.5
    dl = bw.moe_route_backward(logits, idx, w)
    tail = slice(t - 3, t)
    p = torch.softmax(logits[tail].double(), 1)
    c = p.gather(1, idx[tail].long())
    want = -p * c * c
    want.scatter_add_(1, idx[tail].long(), c * c)
    # |dl| <= 1/4: bfloat16's half step 2^-11 and f32's roundings below it
    assert float((dl[tail].double() - want).abs().max()) <= 2.0 ** -10


def test_calls_on_a_raw_stream_handle():
    """A stream given as its handle: temporaries and outputs outlive the call on it."""
    side = torch.cuda.Stream()
    w = weight(96, (), 4096, 4096, 128, False)
    h = bw.q4_upload(*(cuda(t) for t in w))
    x = torch.randn((300, 4096), generator=gen(97)).bfloat16().cuda()
    note("[q4_gemm] raw stream handle")
    want = bw.q4_gemm(h, x)
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):
        got.append(bw.q4_gemm(h, x, stream=side.cuda_stream))
        torch.full((8 << 20,), 7.0, device="cuda")  # would take the workspace's place
    side.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_refusals_on_the_gpu():
    """Wrong types, shapes, orders and overlaps are refused before anything is queued."""
    w = bw.q4_upload(*(cuda(t) for t in weight(98, (), 64, 128, 32, False)))
    x = torch.zeros((4, 128), device="cuda")
    note("[q4] refusals")
    with pytest.raises(TypeError):
        bw.q4_gemm(w, x.double())
    with pytest.raises(TypeError):
        bw.q4_gemm(w, x, torch.zeros((4, 64), device="cuda", dtype=torch.float16))
    with pytest.raises(TypeError):
        bw.q4_gemm(w, x.cpu())
    with pytest.raises(TypeError):
        bw.q4_gemm(w, [1.0])
    with pytest.raises(ValueError):
        bw.q4_gemm(w, x[:, :96])
    with pytest.raises(ValueError):
        bw.q4_gemm(w, torch.zeros((128, 4), device="cuda").T)
    with pytest.raises(ValueError):
        bw.q4_gemm(w, x, torch.zeros((5, 64), device="cuda"))
    with pytest.raises(bw.Tq2Error):
        bw.q4_gemm(w, x.view(-1)[:256].view(2, 128), x.view(-1)[128:256].view(2, 64))
    logits = torch.zeros((4, 8), device="cuda")
    with pytest.raises(TypeError):
        bw.moe_route(logits, 2, bias=torch.zeros(8, device="cuda").half())
    with pytest.raises(ValueError):
        bw.moe_route(logits, 2, idx=torch.zeros((4, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        bw.moe_route_backward(logits, torch.zeros((4, 2), dtype=torch.int64, device="cuda"), torch.zeros((4, 2), device="cuda"))
    with pytest.raises(ValueError):
        bw.q4_moe(x, torch.zeros((4, 2), dtype=torch.int32, device="cuda"), torch.zeros((4, 2), device="cuda"), w, w, w)


def test_example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mixture_layer.py")
    spec = importlib.util.spec_from_file_location("mixture_layer", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    note("[example] mixture layer")
    layer = ex.MixtureLayer(d=256, f=128, experts=16, chosen=4, groups=4, keep=2, seed=1)
    x = torch.randn((50, 256), generator=gen(99)).bfloat16().cuda()
    out = layer(x)
    # the same layer by its formulas in 64 bits, each intermediate rounded as the layer rounds it
    deq = lambda w: bw.q4_dequant(w).double()  # noqa: E731
    h = bw.q4_gemm(layer.w_in, x)
    idx, wts = layer.route(layer.logits(h))
    y = torch.zeros((50, 256), dtype=torch.float64, device="cuda")
    gate, up, down = deq(layer.gate), deq(layer.up), deq(layer.down)
    for t in range(50):
        for j in range(4):
            e = int(idx[t, j])
            g, u = gate[e] @ h[t].double(), up[e] @ h[t].double()
            y[t] += wts[t, j].double() * (down[e] @ (g / (1 + torch.exp(-g)) * u))
    want = y.bfloat16().double() @ deq(layer.w_out).T.contiguous()
    # two bfloat16 roundings (y, out), the same for y's own error, and h in f16: 2^-8 each at most
    assert float((out.double() - want).norm() / want.norm()) <= 3 * 2.0 ** -8
    losses = ex.tune(layer, h, lambda i: torch.full(i.shape, 0.25, device="cuda"), 10, 0.05)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
