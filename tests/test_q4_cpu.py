"""Refusals and sizes of the 4-bit weight and mixture-of-experts calls (no GPU needed).

The C entry points check every argument on the host before a device is looked at; the
binding refuses tensors that are not on the GPU, of another type, shape or order.  The
64-bit references that the GPU tests compare with are pinned here to closed forms.
"""

import ctypes
import math
import os

import pytest
import torch

import bit_weight_gemm_amd as bw
from q4_util import dequant64, gen, moe64, route64, route_weights64, weight


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(bw.LIB_PATH):
        from bit_weight_gemm_amd import build
        build.build()
    return bw.lib()


A = 1 << 20  # an address that is never read: every call below is refused, or ends at the device check


def w4(e=1, n=64, k=128, g=32, zeros=0, data=A):
    s = bw._Q4Struct(data, e, n, k, g, zeros, 0)
    return s


def ptr(s):
    return ctypes.addressof(s)


def test_packed_size(L):
    # head, a kilobyte a unit of 16 rows and 128 k, scales, zero points
    assert L.q4_packed_size(1, 4096, 4096, 128, 0) == 256 + 256 * 32 * 1024 + 256 * 32 * 32
    assert L.q4_packed_size(1, 17, 160, 32, 1) == 256 + 4 * 1024 + 4 * 128 + 4 * 64
    assert L.q4_packed_size(8, 16, 128, 64, 0) == 256 + 8 * 1024 + 8 * 64
    for bad in ((0, 16, 128, 32), (1, 0, 128, 32), (1, 16, 0, 32), (1, 16, 130, 32), (1, 16, 128, 16), (1, 16, 96, 64),
                (1025, 16, 128, 32), (1, (1 << 24) + 1, 128, 32), (1, 16, (1 << 20) + 128, 128), (-1, 16, 128, 32)):
        assert L.q4_packed_size(*bad, 0) == 0, bad


def test_pack_and_dequant_refusals(L):
    bad = bw.TQ2_EINVAL
    w = w4()
    far = A + (1 << 16)
    assert L.q4_pack(None, far, far, None, None) == bad
    assert L.q4_pack(ptr(w), None, far, None, None) == bad
    assert L.q4_pack(ptr(w), far, None, None, None) == bad
    assert L.q4_pack(ptr(w), far, far, far, None) == bad                     # zero points that the weight does not name
    assert L.q4_pack(ptr(w4(zeros=1)), far, far, None, None) == bad
    assert L.q4_pack(ptr(w), far + 2, far, None, None) == bad                # codes not 4-byte aligned
    assert L.q4_pack(ptr(w), A + 512, far, None, None) == bad                # overlap
    assert L.q4_pack(ptr(w4(data=A + 16)), far, far, None, None) == bad      # packed memory not 256-byte aligned
    assert L.q4_pack(ptr(w4(k=100)), far, far, None, None) == bad
    assert L.q4_dequant(ptr(w), None, None) == bad
    assert L.q4_dequant(ptr(w), A + 256, None) == bad
    assert L.q4_dequant(None, far, None) == bad


def test_gemm_refusals(L):
    bad, far, y = bw.TQ2_EINVAL, A + (1 << 16), A + (1 << 18)
    w = w4()
    assert L.q4_gemm(None, far, y, 1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w4(e=2)), far, y, 1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far, y, -1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far, y, 1 << 31, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far, y, 1, 3, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), None, y, 1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far, None, 1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far + 4, y, 1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far, y + 8, 1, 0, None, 0, None) == bad
    assert L.q4_gemm(ptr(w), far, far + 16, 1, 0, None, 0, None) == bad      # y over x
    assert L.q4_gemm(ptr(w), far, A + 512, 1, 0, None, 0, None) == bad       # y over the weight
    for m in (1, 16):
        assert L.q4_gemm_workspace_size(ptr(w), m, 0) == 0
    assert L.q4_gemm_workspace_size(ptr(w), -1, 0) == 0
    big = w4(n=4096, k=4096, g=128)
    need = L.q4_gemm_workspace_size(ptr(big), 2048, bw.Q4_F32)
    if need:
        x, out, ws = A + (1 << 26), A + (1 << 28), A + (1 << 30)
        assert L.q4_gemm(ptr(big), x, out, 2048, bw.Q4_F32, None, 0, None) == bad
        assert L.q4_gemm(ptr(big), x, out, 2048, bw.Q4_F32, ws, need - 1, None) == bad
        assert L.q4_gemm(ptr(big), x, out, 2048, bw.Q4_F32, ws + 64, need, None) == bad
        assert L.q4_gemm(ptr(big), x, out, 2048, bw.Q4_F32, out + 256, need, None) == bad


def test_route_refusals(L):
    bad, l, i, w, b = bw.TQ2_EINVAL, A, A + (1 << 20), A + (1 << 21), A + (1 << 22)

    def call(logits=l, bias=None, idx=i, wts=w, t=4, e=64, k=8, groups=1, keep=1, top=1, score=0, dtype=0):
        return L.moe_route(logits, bias, idx, wts, t, e, k, groups, keep, top, score, 0, dtype, None)

    for kw in (dict(logits=None), dict(idx=None), dict(wts=None), dict(t=-1), dict(t=1 << 31), dict(e=0), dict(e=1025),
               dict(k=0), dict(k=65), dict(e=4, k=5), dict(groups=0), dict(groups=7), dict(groups=128, e=1024),
               dict(groups=8, keep=9), dict(keep=0), dict(top=0), dict(top=3), dict(score=2), dict(score=-1),
               dict(dtype=3), dict(logits=l + 2), dict(logits=l + 1, dtype=1), dict(idx=i + 2), dict(wts=w + 1),
               dict(bias=b + 2), dict(idx=l + 16), dict(wts=l), dict(wts=i + 64), dict(bias=i)):
        assert call(**kw) == bad, kw

    def back(logits=l, idx=i, dw=w, dl=b, t=4, e=64, k=8, score=0, dtype=0):
        return L.moe_route_backward(logits, idx, dw, dl, t, e, k, score, 0, dtype, None)

    for kw in (dict(logits=None), dict(idx=None), dict(dw=None), dict(dl=None), dict(t=-1), dict(e=0), dict(e=1025),
               dict(k=0), dict(k=65), dict(score=5), dict(dtype=-1), dict(dl=l), dict(dl=i), dict(dl=w), dict(dl=b + 2)):
        assert back(**kw) == bad, kw


def test_moe_refusals(L):
    bad = bw.TQ2_EINVAL
    x, i, w, y, ws = A + (1 << 24), A + (1 << 25), A + (1 << 26), A + (1 << 27), A + (1 << 28)
    gate, up, down = w4(4, 64, 128), w4(4, 64, 128, data=A + (1 << 20)), w4(4, 128, 64, data=A + (1 << 21))
    need = L.q4_moe_workspace_size(5, 2, 4, 128, 64, 0)
    assert need > 0

    def call(x=x, i=i, w=w, gate=gate, up=up, down=down, y=y, t=5, k=2, dtype=0, ws=ws, n=need):
        return L.q4_moe(x, i, w, ptr(gate), ptr(up), ptr(down), y, t, k, dtype, ws, n, None)

    for kw in (dict(x=None), dict(i=None), dict(w=None), dict(y=None), dict(t=-1), dict(t=1 << 23), dict(k=0), dict(k=65),
               dict(dtype=7), dict(x=x + 4), dict(y=y + 8), dict(i=i + 1), dict(w=w + 2), dict(y=x), dict(y=i & ~255),
               dict(y=A), dict(y=A + (1 << 20)), dict(ws=None), dict(ws=ws + 128), dict(n=need - 1), dict(ws=y),
               dict(up=w4(4, 96, 128)), dict(up=w4(4, 64, 128, g=64)), dict(up=w4(4, 64, 128, zeros=1)),
               dict(up=w4(3, 64, 128)), dict(down=w4(4, 64, 128)), dict(down=w4(4, 128, 96)), dict(gate=w4(4, 64, 128, data=0)),
               dict(down=w4(2, 128, 64))):
        assert call(**kw) == bad, kw
    for sizes in ((-1, 2, 4, 128, 64, 0), (5, 0, 4, 128, 64, 0), (5, 2, 0, 128, 64, 0), (5, 2, 4, 120, 64, 0),
                  (5, 2, 4, 128, 64, 9), (1 << 23, 2, 4, 128, 64, 0)):
        assert L.q4_moe_workspace_size(*sizes) == 0, sizes


def test_binding_refuses_what_is_not_on_the_gpu():
    codes, scales, zeros = weight(1, (), 16, 64, 32, True)
    with pytest.raises(TypeError):
        bw.q4_upload(codes, scales, zeros)
    with pytest.raises(ValueError):
        bw.q4_upload(codes[0], scales[0])
    with pytest.raises(ValueError):
        bw.q4_upload(codes, scales[:, :0])
    with pytest.raises(ValueError):
        bw.q4_upload(codes, scales.repeat(1, 2))  # G = 16
    logits = torch.zeros((3, 8))
    with pytest.raises(TypeError):
        bw.moe_route(logits, 2)
    with pytest.raises(TypeError):
        bw.moe_route(logits.double(), 2)
    with pytest.raises(ValueError):
        bw.moe_route(logits, 9)
    with pytest.raises(ValueError):
        bw.moe_route(logits, 2, score="tanh")
    with pytest.raises(ValueError):
        bw.moe_route(logits, 2, groups=3)
    with pytest.raises(ValueError):
        bw.moe_route(logits[0], 2)
    with pytest.raises(TypeError):
        bw.moe_route_backward(logits, torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2)))


def test_reference_dequant_by_hand():
    # bytes 0x0F, 0x80: codes 15, 0, 0, 8; zero 8 by default; G covers the row
    codes = torch.zeros((1, 16), dtype=torch.uint8)
    codes[0, 0], codes[0, 1] = 0x0F, 0x80
    scales = torch.tensor([[0.5]]).half()
    got = dequant64(codes, scales, None)[0]
    assert got[:4].tolist() == [3.5, -4.0, -4.0, 0.0] and (got[4:] == -4.0).all()
    got = dequant64(codes, scales, torch.tensor([[3]], dtype=torch.uint8))[0]
    assert got[:4].tolist() == [6.0, -1.5, -1.5, 2.5]


def test_reference_route_by_hand():
    l = torch.log(torch.tensor([[1.0, 2.0, 4.0, 1.0]]))
    idx, w = route64(l, 2, None, "softmax", 1, 1, 1, False)
    assert idx.tolist() == [[2, 1]] and torch.allclose(w, torch.tensor([[0.5, 0.25]], dtype=torch.float64), atol=1e-7)
    idx, w = route64(l, 2, None, "softmax", 1, 1, 1, True)
    assert torch.allclose(w, torch.tensor([[2 / 3, 1 / 3]], dtype=torch.float64), atol=1e-7)
    # two groups, the better by the sum of two: (0.125 + 0.25) against (0.5 + 0.125); equal keys by the lower index
    idx, _ = route64(l, 2, None, "softmax", 2, 1, 2, False)
    assert idx.tolist() == [[2, 3]]
    idx, _ = route64(l, 3, torch.tensor([1.0, 0.0, 0.0, 0.0]), "softmax", 1, 1, 1, False)
    assert idx.tolist() == [[0, 2, 1]]
    l[0, 2] = -math.inf
    idx, w = route64(l, 4, None, "sigmoid", 1, 1, 1, False)
    assert idx.tolist() == [[1, 0, 3, -1]] and w[0, 3] == 0 and abs(float(w[0, 0]) - 2 / 3) < 1e-7


def test_reference_gradient_by_hand():
    """One expert of two: w = p_0, d p_0 / d l = (p0 p1, -p0 p1); renormalised it is 1, without a gradient."""
    l = torch.tensor([[0.3, -0.2]], dtype=torch.float64, requires_grad=True)
    idx = torch.tensor([[0]], dtype=torch.int32)
    p = torch.softmax(l.detach(), 1)[0]
    (g,) = torch.autograd.grad(route_weights64(l, idx, "softmax", False).sum(), l)
    assert torch.allclose(g, torch.tensor([[p[0] * p[1], -p[0] * p[1]]]))
    (g,) = torch.autograd.grad(route_weights64(l, idx, "softmax", True).sum(), l)
    assert torch.allclose(g, torch.zeros(1, 2, dtype=torch.float64), atol=1e-15)


def test_reference_moe_by_hand():
    """d = f = 1: y = sum_j w_j down_e silu(gate_e x) up_e x."""
    one = lambda *v: torch.tensor(v, dtype=torch.float64).view(-1, 1, 1)  # noqa: E731
    x = torch.tensor([[2.0]])
    y = moe64(x, torch.tensor([[1, -1, 0, 2]], dtype=torch.int32), torch.tensor([[0.5, 9.0, 0.25, 9.0]]), one(1.0, -1.0),
              one(3.0, 0.5), one(1.0, 10.0))
    silu = lambda v: v / (1 + math.exp(-v))  # noqa: E731
    assert abs(float(y) - (0.5 * 10 * silu(-2.0) * 1.0 + 0.25 * silu(2.0) * 6.0)) < 1e-12
