"""4-bit products of bfloat16 rows against bounds that leave no room for rounded weights.

Every kernel forms its products exactly (code - zero, or 16 + code, by x's own bits) and sums them in f32, so a
bfloat16 result is off by half a step of bfloat16, 2^-8 of its value, and by the f32 sums: at most (3 G + K/G + 32)
roundings of 2^-24 on partial sums below 62 B, B = sum |x| scale, element by element; in the 2-norm 2^-20 of the result's.

"""

import pytest
import torch

from gpu_util import note
from q4_util import dequant64, gen, weight
from test_gpu_q4 import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 1000, 4096), (16, 4100, 1024), (33, 1040, 2048), (65, 500, 512), (130, 2051, 4096),
                                   (256, 1000, 8192), (700, 2048, 1152), (2050, 4096, 384)])
def test_bfloat16_rows(m, n, k, group):
    codes, scales, zeros = w = weight(1, (), n, k, group, True)
    x = torch.randn((m, k), generator=gen(2)).bfloat16().cuda()
    note(f"[q4_gemm] bounds M={m} N={n} K={k} G={group}")
    y = run(x, w, "bf16").double()
    x64 = x.double()
    want = x64 @ dequant64(*w).cuda().T.contiguous()
    b = x64.abs() @ scales.double().cuda().repeat_interleave(group, -1).T.contiguous()
    err = (y - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + (3 * group + k // group + 32) * 2.0 ** -24 * 62 * b).all()
    rel = float(err.norm() / want.norm())
    note(f"  rel {rel:.3g}")
    # half a step is at most 2^-8 of a value, and independent errors spread evenly over a step are 1/sqrt(3) of that
    assert rel <= 2.0 ** -8 / 3 ** 0.5 + 2.0 ** -20
