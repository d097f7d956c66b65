"""Workspace sizes of the 4-bit products and the compiled calls' refusals, without a GPU."""

import ctypes

import pytest
import torch

import bit_weight_gemm_amd as bw
from test_q4_cpu import L, ptr, w4  # noqa: F401  (L: the fixture)


def up256(v):
    return (v + 255) // 256 * 256


def test_gemm_workspace_sizes(L):
    big = w4(n=4096, k=4096, g=128)
    for dtype in (bw.Q4_F32, bw.Q4_F16, bw.Q4_BF16):
        for m in (0, 1, 16, 32):
            assert L.q4_gemm_workspace_size(ptr(big), m, dtype) == 0
    # one share of the units: planes and row scales (none for f16 rows of whole units)
    assert L.q4_gemm_workspace_size(ptr(big), 2048, bw.Q4_F16) == 0
    assert L.q4_gemm_workspace_size(ptr(big), 2048, bw.Q4_BF16) == 2048 * 4096 * 2 + 2048 * 4
    assert L.q4_gemm_workspace_size(ptr(big), 2048, bw.Q4_F32) == 2 * 2048 * 4096 * 2 + 2048 * 4
    # several shares: f32 sums of each, whole fours of them
    n, m = 4099, 255
    odd = w4(n=n, k=4096, g=128)
    need = L.q4_gemm_workspace_size(ptr(odd), m, bw.Q4_F16)
    share = (m * n + 3) // 4 * 16
    assert need > 0 and need % share == 0 and 2 <= need // share <= 16
    planes = up256(m * 4096 * 2) + up256(m * 4)
    need = L.q4_gemm_workspace_size(ptr(odd), m, bw.Q4_BF16)
    assert need > planes and (need - planes) % share == 0
    # a weight so narrow that blocks of 32 rows would pass a grid's second axis
    narrow = w4(n=16, k=128, g=128)
    assert L.q4_gemm_workspace_size(ptr(narrow), (1 << 31) - 1, bw.Q4_BF16) > 0
    assert L.q4_gemm_workspace_size(ptr(big), 2048, 3) == 0
    assert L.q4_gemm_workspace_size(None, 2048, 0) == 0


def test_moe_workspace_sizes(L):
    for t, k, e, d, f in ((1, 8, 64, 2048, 1024), (8, 8, 64, 2048, 1024), (33, 4, 32, 1024, 1536), (100, 2, 8, 1024, 1024),
                          (2048, 8, 64, 2048, 1024), (0, 4, 8, 128, 128)):
        for dtype in (bw.Q4_F32, bw.Q4_F16, bw.Q4_BF16):
            need = L.q4_moe_workspace_size(t, k, e, d, f, dtype)
            assert need >= 256 + t * k * d * 4, (t, dtype)  # at least each slot's part


def test_compiled_calls_refuse(L):
    calls = bw._calls()
    for f in (calls.gemm, calls.route, calls.route_backward, calls.moe, calls.address, calls.stream, calls.bind):
        with pytest.raises(TypeError):
            f()
    w = w4()
    with pytest.raises(TypeError):
        calls.gemm(ctypes.addressof(w), 0, "x", None, None)
    with pytest.raises(TypeError):
        calls.gemm(ctypes.addressof(w), 0, torch.zeros((1, 128)), None, None)
    with pytest.raises(ValueError):
        calls.gemm(ctypes.addressof(w), 0, torch.zeros(128), None, None)
    with pytest.raises(TypeError):
        calls.route(torch.zeros((2, 8)), "k", None, 0, 1, 1, 1, False, None, None, None)
    with pytest.raises(TypeError):
        calls.address(torch.zeros(4), "f32", (4,), "t", 0)
    with pytest.raises(TypeError):
        bw.moe_route([1.0], 1)
