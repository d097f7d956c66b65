"""The block's calls at narrow widths, far offsets and on other streams' memory.

Tolerances as in the tests of each call.
"""

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import cuda, gen, weight
from test_gpu_linear import check
from test_gpu_streams import pool_of, side_stream

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n", [(40, 1), (300, 5), (300, 7), (130, 8), (257, 9), (1030, 3), (2100, 15)])
def test_linear_of_few_columns(m, n, dtype):
    check(m, n, 1024, 128, True, dtype, "gelu_tanh", "f32", True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [64, 2048])
def test_linear_tiles_of_few_columns(m, dtype):
    """Narrow and deep: many shares of the units, or whole tiles of which most columns are missing."""
    for n in (6, 250, 259):
        check(m, n, 8192, 64, False, dtype, "relu", None, True)


def test_norms_of_rows_past_four_gigabytes():
    """5 GB a tensor: the last rows agree with the same rows alone."""
    m, n = 300000, 8192
    note(f"[block_norm] M={m} N={n}")
    x = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    x[:] = torch.randn((1, n), generator=gen(1)).bfloat16().cuda()
    b = x.clone()
    tail = slice(m - 3, m)
    for t, s in ((x, 2), (b, 3)):
        t[tail] = torch.randn((3, n), generator=gen(s)).bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(n, generator=gen(4))).bfloat16().cuda()
    y, nn = bw.block_norm(x, b=b, post=w, pre=w)
    ys, ns = bw.block_norm(x[tail].clone(), b=b[tail].clone(), post=w, pre=w)
    assert torch.equal(y[tail], ys) and torch.equal(nn[tail], ns)
    out = bw.block_norm_backward(x, y, dn=nn, b=b, post=w, pre=w)
    few = bw.block_norm_backward(x[tail].clone(), ys, dn=ns, b=b[tail].clone(), post=w, pre=w)
    assert torch.equal(out["dx"][tail], few["dx"]) and torch.equal(out["db"][tail], few["db"])


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_come_from_their_streams_pool(raw):
    side = side_stream()
    stream = side.cuda_stream if raw else side
    w = bw.q4_upload(*(cuda(t) for t in weight(1, (4,), 128, 128, 64, True)))
    dense = bw.q4_upload(*(cuda(t) for t in weight(2, (), 128, 128, 64, True)))
    x = torch.randn((8, 128), generator=gen(3)).cuda()
    r, g = torch.randn((4, 128), generator=gen(4)).cuda(), torch.randn(128, generator=gen(5)).cuda()
    torch.cuda.synchronize()
    note(f"[streams] a block's outputs raw={raw}")
    run = lambda s: {"q4_linear": bw.q4_linear(dense, x, bias=g, residual=x, stream=s),  # noqa: E731
                     **dict(zip(("y", "idx", "weights"), bw.moe_layer(x, r, w, w, w, 2, norm=g, residual=x, stream=s))),
                     **dict(zip(("sum", "n"), bw.block_norm(x, b=x, post=g, gate=r[:2], pre=g, stream=s))),
                     **bw.block_norm_backward(x, x, dn=x, b=x, post=g, gate=r[:2], pre=g, stream=s)}
    got = run(stream)
    for what, t in got.items():
        assert pool_of(t) == side.cuda_stream, what
    side.synchronize()
    for what, t in run(None).items():
        assert torch.equal(got[what], t), what


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,k,masked", [(1, 1, False), (2, 3, True), (2, 16, False), (4, 8, False), (3, 9, True)])
def test_layer_of_a_few_tokens_in_one_launch(t, k, masked, dtype):
    """Against the reference, with patience and without any: the same bits."""
    from test_gpu_layer import call, check as check_layer, inputs

    x, r, w, a = inputs(t, 24, 288, 160, 32, True, dtype, bias=True)
    if masked:
        a["bias"][5:] = -float("inf")
    got = check_layer(x, r, w, k, a, dtype, "few", score="sigmoid", renorm=True)
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    was = bw.moe_layer_set_patience(0)
    try:
        for _ in range(4):
            again = call(x, r, handles, k, a, score="sigmoid", renorm=True)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, again))
    finally:
        bw.moe_layer_set_patience(was)
