"""GPU: the norms and their gradient at rows far from zero, of any size, and constant ones.

Forward tolerances as in test_gpu_block_norm.py, and what a mean far from zero costs in 64 bits: it is a sum of N values over
threads (at most 32 of a thread, six exchanges, eight waves: below 64 roundings of 2^-53), so a normed value is off by at most 64 2^-53
of mean / deviation, here and in the reference each.  Gradient: test_gpu_block_norm.py's.
"""

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import d64, half_step, hat64, least, norm64
from gpu_util import note
from q4_util import gen
from test_gpu_block_norm import check_backward, inputs

pytestmark = pytest.mark.gpu


def check(a, dtype, kind, eps, scale=0.5):
    """y and n against 64 bits, and the gradient at that y."""
    m, n = a["x"].shape
    y, nn = bw.block_norm(a["x"], b=a["b"], post=a["post"], post_bias=a["post_bias"], gate=a["gate"], scale=scale, pre=a["pre"],
                          pre_bias=a["pre_bias"], kind=kind, eps=eps)
    torch.cuda.synchronize()
    w = {k: d64(v) for k, v in a.items()}

    def far(v):
        """mean / deviation of rows, in the roundings of a mean."""
        c = v - v.mean(1, keepdim=True)
        return 128 * 2.0 ** -53 * v.abs().mean(1, keepdim=True) / ((c * c).mean(1, keepdim=True) + eps).sqrt() if kind == "layer" else 0.0

    add = scale * w["gate"] * norm64(w["b"], kind, eps, w["post"], w["post_bias"])
    want = w["x"] + add
    tol = 4 * 2.0 ** -24 * (add.abs() + w["x"].abs()) + (scale * w["gate"] * w["post"]).abs() * far(w["b"])
    tol = tol + half_step(dtype) * want.abs() * 1.01 + least(dtype)
    err = (y.double() - want).abs()
    note(f"  y worst err/tol {float((err / tol).max()):.3g}")
    assert (err <= tol).all()
    want = norm64(y.double(), kind, eps, w["pre"], w["pre_bias"])
    tol = (2.0 ** -23 + half_step(dtype)) * want.abs() + w["pre"].abs() * far(y.double()) + least(dtype)
    err = (nn.double() - want).abs()
    note(f"  n worst err/tol {float((err / tol).max()):.3g}")
    assert (err <= tol).all()
    check_backward(a, y, m, n, dtype, kind, scale, eps=eps)


@pytest.mark.parametrize("m,n", [(6, 60), (5, 250), (4, 500), (9, 1111), (7, 4096), (3, 9001), (2, 16384)])
@pytest.mark.parametrize("log_ratio", [10, 13, 16, 18, 20])
def test_means_far_from_zero(log_ratio, m, n):
    """Deviations of 1 (b) and 2 (x) around a mean of 2^log_ratio, of either sign."""
    a = inputs(m, n, "f32", "layer", True, True, 1, offset=2.0 ** log_ratio)
    a["b"][0] *= -1
    note(f"[block_norm] far rows M={m} N={n} 2^{log_ratio}")
    check(a, "f32", "layer", 1e-6)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [264, 4096, 6001])
def test_means_far_from_zero_in_16_bits(n, dtype):
    """Rows of two neighbouring values of the type: a mean of 2^11 or 2^8 deviations and more."""
    a = inputs(6, n, dtype, "layer", True, True, 1)
    step = 1.0 if dtype == "f16" else 8.0  # of 1024 .. 2047
    for i, v in enumerate((a["x"], a["b"])):
        v.copy_(1500 // step * step + step * (torch.rand(v.shape, generator=gen(30 + i)) < 0.5))
    note(f"[block_norm] far rows N={n} {dtype}")
    check(a, dtype, "layer", 1e-6)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("n", [60, 500, 4096, 9001])
def test_rows_of_any_size(n, kind):
    """Rows of zeros, constant ones, of 1e30 and of 1e-30, and means of 2000 deviations."""
    a = inputs(12, n, "f32", kind, True, True, 1, offset=2000.0)
    for v in (a["x"], a["b"]):
        v[1] = 0
        v[2] = 3.5
        v[3] = 1e30 * (v[3] - 2000)
        v[4] = 1e-30 * (v[4] - 2000)
        v[7] = 0.1
    a["x"][6] = -a["b"][6]
    note(f"[block_norm] rows of any size N={n} {kind}")
    check(a, "f32", kind, 1e-5)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_without_a_finite_statistic(kind):
    """An infinity or NaN makes its own row NaN (with its gradient) and no other."""
    m, n = 40, 1000
    a = inputs(m, n, "f32", kind, True, True, 1, offset=2.0 ** 14)
    call = lambda: bw.block_norm(a["x"], b=a["b"], post=a["post"], post_bias=a["post_bias"], gate=a["gate"], pre=a["pre"],  # noqa: E731
                                 pre_bias=a["pre_bias"], kind=kind)
    clean = call()
    a["b"][3, 5], a["x"][7, 999], a["b"][11, 0] = float("nan"), float("nan"), float("inf")
    note(f"[block_norm] rows without a statistic {kind}")
    y, nn = call()
    rest = [i for i in range(m) if i not in (3, 7, 11)]
    assert torch.equal(y[rest], clean[0][rest]) and torch.equal(nn[rest], clean[1][rest])
    assert torch.isnan(nn[[3, 7]]).all() and torch.isnan(nn[11]).any()
    assert torch.equal(torch.isnan(nn), torch.isnan(norm64(y.double(), kind, 1e-6, d64(a["pre"]), d64(a["pre_bias"]))))
    dn = torch.randn((m, n), generator=gen(9)).cuda()
    one = lambda y: bw.block_norm_backward(None, y, dn=dn, pre=a["pre"], pre_bias=a["pre_bias"], kind=kind)["dx"]  # noqa: E731
    assert torch.equal(one(y)[rest], one(clean[0])[rest]) and torch.isnan(one(y)[[3, 7]]).all()
    assert not torch.isnan(hat64(clean[0].double(), kind, 1e-6)).any()
