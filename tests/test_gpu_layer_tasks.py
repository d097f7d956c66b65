"""GPU: a mixture layer of a few tokens: more pieces of work than workgroups, without patience, masks, mixed group sizes.

Weights in groups of 128 have one launch behind the logits, of at most 512 workgroups; a call with more gate, up and down products
than that gives several to each, in the same LDS.  Other groups have several launches.  Tolerances as in test_gpu_layer.py.
"""

import pytest
import torch

import bit_weight_gemm_amd as bw
from block_util import half_step, layer64
from gpu_util import note
from q4_util import cuda, gen, weight
from test_gpu_layer import call, check, inputs

pytestmark = pytest.mark.gpu


def pieces(t, k, d, f):
    """Gate and up products of 32 columns of a slot, down products of 16 columns of a token."""
    return t * (k * -(-f // 32) + -(-d // 16))


def mixed(e, d, f, up_group, down_group, zeros, seed=1):
    return [weight(seed, (e,), f, d, up_group, zeros), weight(seed + 1, (e,), f, d, up_group, zeros), weight(seed + 2, (e,), d, f, down_group, not zeros)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t,k,d,f,up_group,down_group,residual", [(2, 8, 2048, 1024, 128, 128, True), (4, 8, 2048, 1024, 128, 128, False),
                                                                 (2, 16, 1024, 512, 128, 128, True), (3, 9, 1536, 640, 128, 128, False),
                                                                 (1, 8, 8192, 1024, 128, 128, True), (1, 16, 256, 512, 128, 128, True),
                                                                 (2, 8, 1024, 1024, 128, 64, True), (4, 8, 2048, 1024, 32, 128, False),
                                                                 (3, 9, 1568, 736, 32, 32, False)])
def test_more_work_than_workgroups(t, k, d, f, up_group, down_group, residual, dtype):
    """(One of fewer pieces among them.)  With patience and without: the same bits."""
    e = k + 2
    assert (pieces(t, k, d, f) > 512) == (d > 256)
    x, r, _, a = inputs(t, e, d, 64, 32, False, dtype, residual=residual)
    w = mixed(e, d, f, up_group, down_group, t % 2 == 0)
    got = check(x, r, w, k, a, dtype, f"{pieces(t, k, d, f)} pieces", renorm=True)
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    was = bw.moe_layer_set_patience(0)
    try:
        for _ in range(3):
            again = call(x, r, handles, k, a, renorm=True)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, again))
    finally:
        bw.moe_layer_set_patience(was)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("router", ["plain", "masked", "groups", "all masked"])
@pytest.mark.parametrize("t,k,d,f", [(1, 1, 128, 128), (2, 3, 256, 128), (1, 24, 256, 256), (2, 16, 384, 128), (4, 8, 256, 384)])
def test_few_tokens(t, k, d, f, router, dtype):
    """Groups of 128 and zero points; tokens with fewer experts than slots, or none."""
    x, r, w, a = inputs(t, 24, d, f, 128, True, dtype, norm="f32" if t == 2 else "own", bias=router != "plain")
    kw = dict(score="sigmoid", renorm=True)
    if "masked" in router:
        a["bias"][0 if router == "all masked" else 5:] = -float("inf")
    if router == "groups":
        kw.update(groups=8, keep=4, group_top=2)
    got = check(x, r, w, k, a, dtype, "few " + router, **kw)
    if router == "all masked":
        assert (got[1] == -1).all() and torch.equal(got[0].cpu(), a["residual"])
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    was = bw.moe_layer_set_patience(0)
    try:
        again = call(x, r, handles, k, a, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, again))
    finally:
        bw.moe_layer_set_patience(was)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t,k,d,f,group", [(1, 8, 512, 256, 128), (2, 8, 1024, 512, 128), (4, 8, 256, 384, 128), (1, 8, 512, 256, 64), (3, 4, 288, 96, 32)])
def test_few_tokens_keep_more_than_16_bits(t, k, d, f, group, dtype):
    """silu(g) u is in two bfloat16 parts: 2^-17 of the experts' part of a row, f32 sums 2^-18, and one rounding of the result."""
    x, r, w, a = inputs(t, 12, d, f, group, True, dtype, residual=False)
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    note(f"[moe_layer] T={t} k={k} G={group} {dtype}")
    y, idx, _ = call(x, r, handles, k, a, renorm=True)
    want, want_i, _, _ = layer64(x, r, *w, k, **a, renorm=True)
    assert torch.equal(idx.cpu(), want_i)
    rest = (y.cpu().double() - want).abs() - half_step(dtype) * want.abs() * 1.01  # beyond the result's own rounding
    assert (rest.clamp(min=0).norm(dim=1) <= (2.0 ** -17 + 2.0 ** -18) * want.norm(dim=1)).all()


@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("t", [1, 4])
def test_finer_groups_take_about_as_long(t, group):
    """They have the same codes to read: within half as much again of groups of 128 (one launch for them took 1.2 to 2.6 times
    as long)."""
    k, d, f, e = 8, 2048, 1024, 64
    x, r, _, a = inputs(t, e, d, 64, 32, False, "bf16")
    x, r, a = x.cuda(), r.cuda(), {n: cuda(v) for n, v in a.items()}
    note(f"[moe_layer] groups of {group} and of 128, T={t}")
    best = {}
    for g in (group, 128):
        handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in mixed(e, d, f, g, g, False)]
        bw.moe_layer(x, r, *handles, k, **a)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                bw.moe_layer(x, r, *handles, k, **a)
        times = []
        for _ in range(6):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end) / 20)
        best[g] = min(times)
    note(f"  {1e3 * best[group]:.1f} and {1e3 * best[128]:.1f} us")
    assert best[group] <= 1.5 * best[128]


def test_more_work_than_workgroups_in_a_graph():
    """Replays with new rows: what the fill before them left, and nothing of the replay before."""
    t, k, d, f = 2, 8, 2048, 1024
    x, r, _, a = inputs(t, 10, d, 64, 32, False, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in mixed(10, d, f, 128, 128, True)]
    x, r, a = x.cuda(), r.cuda(), {n: cuda(v) for n, v in a.items()}
    note("[moe_layer] graph of several pieces a workgroup")
    bw.moe_layer(x, r, *handles, k, **a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bw.moe_layer(x, r, *handles, k, **a)
    for rep in range(4):
        x.copy_(3 * torch.randn(x.shape, generator=gen(60 + rep)))
        graph.replay()
        torch.cuda.synchronize()
        want = bw.moe_layer(x, r, *handles, k, **a)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), rep


def test_without_patience_a_workgroup_forms_it_itself():
    """One token whose workgroups all start at once: without patience those of the down products find silu(g) u missing and
    form all of it, 128 times the work, which shows in the time (the bits are the same)."""
    t, k, d, f = 1, 8, 2048, 1024
    assert pieces(t, k, d, f) <= 512
    x, r, _, a = inputs(t, 16, d, 64, 32, False, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in mixed(16, d, f, 128, 128, False)]
    x, r, a = x.cuda(), r.cuda(), {n: cuda(v) for n, v in a.items()}
    note("[moe_layer] without patience")

    def best():
        times = []
        for _ in range(8):
            start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            start.record()
            out = bw.moe_layer(x, r, *handles, k, **a)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        return out, min(times)

    want, patient = best()
    was = bw.moe_layer_set_patience(0)
    try:
        got, hasty = best()
    finally:
        bw.moe_layer_set_patience(was)
    note(f"  {1e3 * patient:.0f} us, without patience {1e3 * hasty:.0f}")
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert hasty > 3 * patient


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1, 2])
@pytest.mark.parametrize("e,k,groups", [(1, 1, 1), (3, 3, 1), (65, 7, 1), (130, 16, 1), (256, 8, 8), (257, 8, 1), (1024, 8, 1), (66, 4, 33)])
def test_numbers_of_experts_of_a_few_tokens(e, k, groups, t, dtype):
    """A lane of the router has one expert, or up to four; beyond 256 experts the router has a launch of its own."""
    x, r, w, a = inputs(t, e, 256, 128, 128, False, dtype, norm=None if t == 2 else "own", bias=True, residual=t == 2)
    check(x, r, w, k, a, dtype, "experts", renorm=True, groups=groups, keep=max(1, groups // 2), group_top=2 if groups > 1 else 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t", [1, 2, 4])
def test_rows_of_a_few_tokens_that_are_not_finite(t, dtype):
    """A NaN row stays alone; an expert whose weights make silu(g) u infinite or NaN shows in the tokens that have it."""
    e, k, d, f = 12, 8, 256, 256
    x, r, w, a = inputs(t, e, d, f, 128, False, dtype)
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    clean = call(x, r, handles, k, a)
    bad = x.clone()
    bad[t - 1, 3] = float("nan")
    note(f"[moe_layer] not finite T={t} {dtype}")
    got = call(bad, r, handles, k, a)
    torch.cuda.synchronize()
    assert torch.isnan(got[0][t - 1]).all()
    assert all(torch.equal(p[: t - 1], q[: t - 1]) for p, q in zip(got, clean))
    for value in (float("inf"), float("nan")):
        w[1][1][5, :, 0] = value  # expert 5's up weights
        broken = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
        y, idx, _ = call(x, r, broken, k, a)
        torch.cuda.synchronize()
        has = (idx == 5).any(1)
        assert torch.equal(idx, clean[1]) and torch.isfinite(y[~has]).all() and not torch.isfinite(y[has]).any()
        was = bw.moe_layer_set_patience(0)
        try:
            again, _, _ = call(x, r, broken, k, a)
            torch.cuda.synchronize()
        finally:
            bw.moe_layer_set_patience(was)
        assert torch.equal(torch.isnan(again), torch.isnan(y)) and torch.equal(again[~torch.isnan(y)], y[~torch.isnan(y)])


def test_calls_of_a_few_tokens_side_by_side():
    """Many calls on three streams at once beside a long product, each with a workspace of its own."""
    x, r, w, a = inputs(8, 16, 1024, 512, 128, True, "bf16")
    handles = [bw.q4_upload(*(cuda(v) for v in p)) for p in w]
    x, r, a = x.cuda(), r.cuda(), {k: cuda(v) for k, v in a.items()}
    cuts = ((0, 1), (1, 2), (3, 1), (4, 4))
    rows = [x[i: i + n].contiguous() for i, n in cuts]
    res = [a["residual"][i: i + n].contiguous() for i, n in cuts]
    one = lambda i, s=None: bw.moe_layer(rows[i], r, *handles, 8, norm=a["norm"], residual=res[i], stream=s)  # noqa: E731
    want = [one(i) for i in range(4)]
    big = bw.q4_upload(*(cuda(v) for v in weight(70, (), 4096, 4096, 128, False)))
    wide = torch.randn((4096, 4096), generator=gen(71)).bfloat16().cuda()
    torch.cuda.synchronize()
    note("[moe_layer] a few tokens on three streams")
    # (torch hands out 32 streams in turn: a whole round leaves the turn, on which other tests' fresh streams depend, where it was)
    streams = [torch.cuda.Stream() for _ in range(32)][:4]
    got = []
    for i in range(48):
        if i % 8 == 0:
            bw.q4_gemm(big, wide, stream=streams[3])
        got.append((i % 4, one(i % 4, streams[i % 3])))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(p, q) for p, q in zip(out, want[i]))
