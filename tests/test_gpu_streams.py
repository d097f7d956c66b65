"""Calls on a stream that is not the current one: whose memory their outputs and workspaces are.

A call's kernels write its output and its workspace as soon as `stream` reaches them.  Memory of the current
stream's pool may still be in use by work that is queued there, so both have to come from the pool of `stream`:
every test looks at the allocator's own record of the segment that an address lies in.
"""

import pytest
import torch

import bit_weight_gemm_amd as bw
import workloads as wl
from gpu_util import bits_dev, note, to_dev
from q4_util import cuda, gen, weight

pytestmark = pytest.mark.gpu


def pool_of(t):
    """Handle of the stream whose pool the tensor's memory belongs to."""
    at = t.data_ptr()
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= at < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("no segment holds the tensor")


def pool_bytes(handle):
    return sum(s["total_size"] for s in torch.cuda.memory_snapshot() if s["stream"] == handle)


def side_stream():
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return torch.cuda.Stream()


@pytest.mark.parametrize("raw", [False, True])
def test_new_calls_outputs_come_from_their_streams_pool(raw):
    side = side_stream()
    stream = side.cuda_stream if raw else side
    codes, scales, zeros = (cuda(t) for t in weight(1, (4,), 128, 128, 64, True))
    x = torch.randn((8, 128), generator=gen(2)).cuda()
    idx = torch.randint(0, 4, (8, 2), generator=gen(3)).int().cuda()
    wts = torch.rand((8, 2), generator=gen(4)).cuda()
    logits = torch.randn((8, 4), generator=gen(5)).cuda()
    torch.cuda.synchronize()
    note(f"[streams] outputs raw={raw}")
    w = bw.q4_upload(codes, scales, zeros, stream=stream)
    dense = bw.q4_upload(codes[0], scales[0], zeros[0], stream=stream)
    got = {"packed weight": w.data, "q4_dequant": bw.q4_dequant(w, stream=stream),
           "q4_gemm": bw.q4_gemm(dense, x, stream=stream),
           "q4_moe": bw.q4_moe(x, idx, wts, w, w, w, stream=stream),
           "moe_route_backward": bw.moe_route_backward(logits, idx, wts, stream=stream)}
    got["moe_route idx"], got["moe_route weights"] = bw.moe_route(logits, 2, stream=stream)
    for what, t in got.items():
        assert pool_of(t) == side.cuda_stream, what
    side.synchronize()
    assert torch.equal(got["q4_gemm"], bw.q4_gemm(dense, x)) and torch.equal(got["q4_moe"], bw.q4_moe(x, idx, wts, w, w, w))


def test_new_calls_workspaces_come_from_their_streams_pool():
    side = side_stream()
    n, k, m = 4096, 4096, 300
    w = bw.q4_upload(*(cuda(t) for t in weight(6, (), n, k, 128, False)))
    x = torch.randn((m, k), generator=gen(7)).bfloat16().cuda()
    y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    need = bw.lib().q4_gemm_workspace_size(w.handle, m, bw.Q4_BF16)
    assert need > 4 << 20
    torch.cuda.synchronize()
    note("[streams] workspace of q4_gemm")
    bw.q4_gemm(w, x, y, stream=side)
    assert pool_bytes(side.cuda_stream) >= need
    side.synchronize()
    assert torch.equal(y, bw.q4_gemm(w, x))

    side = side_stream()
    t, e, k, d, f = 512, 8, 2, 1024, 512
    gate, up, down = (bw.q4_upload(*(cuda(t) for t in weight(8 + i, (e,), *s, 128, False)))
                      for i, s in enumerate(((f, d), (f, d), (d, f))))
    x = torch.randn((t, d), generator=gen(12)).bfloat16().cuda()
    idx = torch.randint(0, e, (t, k), generator=gen(13)).int().cuda()
    wts = torch.rand((t, k), generator=gen(14)).cuda()
    y = torch.empty_like(x)
    need = bw.lib().q4_moe_workspace_size(t, k, e, d, f, bw.Q4_BF16)
    assert need > 4 << 20
    torch.cuda.synchronize()
    note("[streams] workspace of q4_moe")
    bw.q4_moe(x, idx, wts, gate, up, down, y, stream=side)
    assert pool_bytes(side.cuda_stream) >= need
    side.synchronize()
    assert torch.equal(y, bw.q4_moe(x, idx, wts, gate, up, down))


def test_memory_that_the_current_stream_still_uses_is_left_alone():
    """A tensor is read by work queued on the current stream, then freed; a call on another stream may not take its place."""
    side = side_stream()
    n, k, m = 4096, 4096, 300
    w = bw.q4_upload(*(cuda(t) for t in weight(15, (), n, k, 128, False)))
    x = torch.randn((m, k), generator=gen(16)).bfloat16().cuda()
    want = bw.q4_gemm(w, x)
    size = bw.lib().q4_gemm_workspace_size(w.handle, m, bw.Q4_BF16)
    keep = torch.empty(size, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    note("[streams] memory in use by the current stream")
    held = torch.full((size,), 7, dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(200_000_000)
    torch.add(held, 0, out=keep)
    del held
    got = bw.q4_gemm(w, x, stream=side)
    torch.cuda.synchronize()
    assert (keep == 7).all() and torch.equal(got, want)


def test_an_output_is_kept_for_the_callers_stream():
    """The result is read by the current stream and dropped: its memory waits for that."""
    side = side_stream()
    n, k, m = 4096, 1024, 256
    w = bw.q4_upload(*(cuda(t) for t in weight(17, (), n, k, 128, False)))
    x = torch.randn((m, k), generator=gen(18)).half().cuda()
    keep, minus, want = torch.empty((m, n), dtype=torch.float16, device="cuda"), -x, bw.q4_gemm(w, x)
    torch.cuda.synchronize()
    note("[streams] an output on the caller's stream")
    got = bw.q4_gemm(w, x, stream=side)
    at = got.data_ptr()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(200_000_000)
    torch.neg(got, out=keep)
    done = torch.cuda.Event()
    done.record()
    del got
    other = bw.q4_gemm(w, minus, stream=side)
    assert other.data_ptr() != at or done.query()
    torch.cuda.synchronize()
    assert torch.equal(-keep, want)


def new_calls():
    """Each 4-bit or mixture call on a stream, as (name, call(stream, tensors), tensors of its arguments)."""
    codes, scales, zeros = (cuda(t) for t in weight(20, (4,), 128, 128, 64, True))
    w = lambda: bw.q4_upload(codes, scales, zeros)  # noqa: E731
    dense = lambda: bw.q4_upload(codes[0], scales[0], zeros[0])  # noqa: E731
    x = lambda: torch.randn((300, 128), generator=gen(21)).cuda()  # noqa: E731
    idx = lambda: torch.randint(0, 4, (300, 2), generator=gen(22)).int().cuda()  # noqa: E731
    wts = lambda: torch.rand((300, 2), generator=gen(23)).cuda()  # noqa: E731
    logits = lambda: torch.randn((300, 4), generator=gen(24)).cuda()  # noqa: E731
    return [("q4_upload", lambda s, a: bw.q4_upload(*a, stream=s), [codes.clone(), scales.clone(), zeros.clone()]),
            ("q4_dequant", lambda s, a: bw.q4_dequant(a[0], stream=s), [w()]),
            ("q4_gemm", lambda s, a: bw.q4_gemm(*a, stream=s), [dense(), x()]),
            ("moe_route", lambda s, a: bw.moe_route(a[0], 2, bias=a[1], stream=s), [logits(), torch.zeros(4, device="cuda")]),
            ("moe_route_backward", lambda s, a: bw.moe_route_backward(*a, stream=s), [logits(), idx(), wts()]),
            ("q4_moe", lambda s, a: bw.q4_moe(*a, stream=s), [x(), idx(), wts(), w(), w(), w()])]


def test_arguments_may_be_freed_at_once():
    """Memory of a call's arguments is not handed out again before its stream is done with it."""
    side = side_stream()
    calls = new_calls()
    torch.cuda.synchronize()
    for what, call, args in calls:
        note(f"[streams] arguments of {what}")
        data = [a.data if isinstance(a, bw.Q4Weight) else a for a in args]
        places = [(t.data_ptr(), t.numel() * t.element_size()) for t in data]
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        out = call(side, args)
        done = torch.cuda.Event()
        done.record(side)
        del data
        args.clear()
        again = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in places]
        assert not {at for at, _ in places} & {t.data_ptr() for t in again} or done.query(), what
        side.synchronize()
        del out


@pytest.mark.parametrize("raw", [False, True])
def test_ternary_and_blr_calls_memory_comes_from_their_streams_pool(raw):
    side = side_stream()
    stream = side.cuda_stream if raw else side
    aos, n, k = wl.tiny_weight()
    m, d_in, d_out, r = 64, 1024, 1024, 512
    d = wl.blr_inputs(m=m, d_in=d_in, d_out=d_out, r=r, index=60)
    one = [bits_dev(d["bits_u"]), bits_dev(d["bits_v"])] + [to_dev(d[v]) for v in ("h", "l", "g", "x")]
    paths = [t[None].contiguous() for t in one[:5]] + one[5:]
    x = to_dev(wl.tiny_x(5, k))
    dy = 1e-3 * torch.randn((m, d_out), generator=gen(19)).cuda()
    zero = lambda: [torch.zeros((1, v), device="cuda") for v in (d_out, r, d_in)]  # noqa: E731
    grads = [zero() for _ in range(3)]
    torch.cuda.synchronize()
    note(f"[streams] ternary and BLR calls raw={raw}")
    w = bw.tq2_upload(aos, n, k, stream=stream)
    try:
        got = {"tq2_gemm": bw.tq2_gemm(w, x, stream=stream), "tq2_dequant": bw.tq2_dequant(w, stream=stream)}
        got["blr_forward_ws"] = bw.blr_forward_ws(*one, stream=stream)
        got["blr_forward_paths"] = bw.blr_forward_paths(*paths, stream=stream)
        y, saved = bw.blr_forward_paths_save(*paths, stream=stream)
        got["blr_forward_paths_save y"], got["saved"] = y, saved
        got["blr_backward_paths"] = bw.blr_backward_paths(*paths, dy, *grads[0], stream=stream)
        got["blr_backward_paths_saved"] = bw.blr_backward_paths_saved(*paths, dy, *grads[1], saved, stream=stream)
        got["blr_backward_paths_ws"] = bw.blr_backward_paths_ws(*paths, dy, *grads[2], stream=stream)
        for what, t in got.items():
            assert pool_of(t) == side.cuda_stream, what
        side.synchronize()
        assert torch.equal(got["tq2_gemm"], bw.tq2_gemm(w, x))
        assert torch.equal(got["blr_forward_ws"], bw.blr_forward(*one))
        assert torch.equal(got["blr_backward_paths"], got["blr_backward_paths_ws"])
    finally:
        torch.cuda.synchronize()
        w.close()


def test_a_workspace_of_blr_comes_from_its_streams_pool():
    side = side_stream()
    m, d_in, d_out, r = 256, 4096, 1024, 1024
    d = wl.blr_inputs(m=m, d_in=d_in, d_out=d_out, r=r, index=61)
    one = [bits_dev(d["bits_u"]), bits_dev(d["bits_v"])] + [to_dev(d[v]) for v in ("h", "l", "g", "x")]
    y = torch.empty((m, d_out), device="cuda")
    need = bw.blr_workspace_size(m, d_in, d_out, r)
    torch.cuda.synchronize()
    note("[streams] workspace of blr_forward_ws")
    bw.blr_forward_ws(*one, y, stream=side)
    assert need > 0 and pool_bytes(side.cuda_stream) >= need
    side.synchronize()
    assert torch.equal(y, bw.blr_forward(*one))
