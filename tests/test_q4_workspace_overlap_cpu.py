"""A workspace that lies over an input of its call is refused before a device is looked at (no GPU needed)."""

import bit_weight_gemm_amd as bw
from test_q4_cpu import A, L, ptr, w4  # noqa: F401  (L: the fixture)


def test_gemm(L):
    big = w4(n=4096, k=4096, g=128)
    need = L.q4_gemm_workspace_size(ptr(big), 2048, bw.Q4_F32)
    x, y = A + (1 << 26), A + (1 << 28)
    for ws in (x, x + (1 << 24), x - need + 256, A, A + (1 << 20)):
        assert L.q4_gemm(ptr(big), x, y, 2048, bw.Q4_F32, ws, need, None) == bw.TQ2_EINVAL, ws - A


def test_moe(L):
    at = [A + (i << 24) for i in range(8)]
    gate, up, down = w4(4, 64, 128, data=at[0]), w4(4, 64, 128, data=at[1]), w4(4, 128, 64, data=at[2])
    x, i, w, y = at[3:7]
    for t, dtype in ((5, bw.Q4_F32), (600, bw.Q4_BF16)):
        need = L.q4_moe_workspace_size(t, 2, 4, 128, 64, dtype)
        for ws in (*at[:7], x - need + 256, i - need + 256, w - need + 256):
            assert L.q4_moe(x, i, w, ptr(gate), ptr(up), ptr(down), y, t, 2, dtype, ws, need, None) == bw.TQ2_EINVAL
