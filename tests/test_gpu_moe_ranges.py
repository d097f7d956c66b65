"""Experts' products over weights and activations of very different size, from one token to long prompts.

Long prompts hold silu(g) u of 16-bit types in f16 under powers of two.  What must not depend on those powers: groups
of large scale whose codes are all the zero point, single large weights, zero points of a whole byte, and rows near
both ends of bfloat16.  Token counts here take every deal: single slots, slots that workgroups find, blocks of
16 rows, tiles of 64 and of 128.

Tolerances, in the norm of each token's row: the result's rounding, half a step (eps/2); silu(g) u's rounding to
f16, 2^-11 of each term, whose errors are independent, so 2^-11 of a sum's norm covers sqrt(3) times their own; f32 sums 2^-18.
"""

import pytest
import torch

import bit_weight_gemm_amd as bw
from gpu_util import note
from q4_util import DTYPES, cuda, dequant64, gen, weight

pytestmark = pytest.mark.gpu

E, K, D, F = 16, 2, 256, 256
TOKENS = [1, 16, 20, 120, 400, 2100]


def tolerance(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2 + 2.0 ** -18 + (0 if dtype == "f32" else 2.0 ** -11)


def layer(seed, zeros=False, group=64):
    return [weight(seed, (E,), F, D, group, zeros), weight(seed + 1, (E,), F, D, group, zeros),
            weight(seed + 2, (E,), D, F, group, zeros)]


def choice(seed, t):
    idx = torch.stack([torch.randperm(E, generator=gen(seed + i))[:K] for i in range(t)]).int()
    return idx, torch.rand((t, K), generator=gen(seed)) + 0.1


def exact(x, idx, wts, w):
    """The layer from its formula in f64, expert by expert."""
    gate, up, down = (dequant64(*v).cuda() for v in w)
    x, idx, wts = x.double().cuda(), idx.cuda(), wts.double().cuda()
    y = torch.zeros((x.shape[0], down.shape[1]), dtype=torch.float64, device="cuda")
    for e in range(gate.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        if len(t):
            g, u = x[t] @ gate[e].T.contiguous(), x[t] @ up[e].T.contiguous()
            h = g / (1 + torch.exp(-g)) * u
            y.index_add_(0, t, (h @ down[e].T.contiguous()) * wts[t, j][:, None])
    return y


def check(x, idx, wts, w, dtype, what):
    note(f"[q4_moe {what}] T={x.shape[0]} {dtype}")
    y = bw.q4_moe(x.cuda(), idx.cuda(), wts.cuda(), *(bw.q4_upload(*(cuda(t) for t in v)) for v in w)).double()
    want = exact(x, idx, wts, w)
    assert torch.isfinite(y).all(), what
    rel = float(((y - want).norm(dim=1) / want.norm(dim=1)).max())
    note(f"  worst row {rel:.3g} (allowed {tolerance(dtype):.3g})")
    assert rel <= tolerance(dtype), what


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("scale", [1.0, 64.0])
def test_groups_that_are_all_zero_point_do_not_count(scale, t, dtype):
    """One group of codes 8 (weight 0) under a large scale in gate and in up, as quantisers leave for empty groups."""
    w = layer(1)
    for codes, scales, _ in w[:2]:
        codes[:, 3, :32] = 0x88
        scales[:, 3, 0] = scale
    x = torch.randn((t, D), generator=gen(5)).to(DTYPES[dtype])
    check(x, *choice(6, t), w, dtype, f"empty group of scale {scale}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("times", [30, 1000])
def test_single_large_rows_of_gate_and_up(times, t, dtype):
    """A row of gate and of up much larger than the others, whose group in down has scale 0: the others keep their bits."""
    w = layer(11)
    for _, scales, _ in w[:2]:
        scales[:, 7] = (scales[:, 7].float() * times).half()
    w[2][1][:, :, 0] = 0
    x = torch.randn((t, D), generator=gen(15)).to(DTYPES[dtype])
    check(x, *choice(16, t), w, dtype, f"rows {times} times as large")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("t", TOKENS)
def test_zero_points_of_a_whole_byte(t, dtype):
    """Rows of -1 against codes 0 under zero points 255: every term of every sum has one sign."""
    n = lambda n, k, s: (torch.zeros((E, n, k // 2), dtype=torch.uint8), torch.full((E, n, k // 128), s).half(),  # noqa: E731
                         torch.full((E, n, k // 128), 255, dtype=torch.uint8))
    w = [n(128, 128, 0.01), n(128, 128, 0.01), n(128, 128, 2.0 ** -20)]
    x = torch.full((t, 128), -1.0).to(DTYPES[dtype])
    check(x, *choice(21, t), w, dtype, "zero points 255")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t", TOKENS)
@pytest.mark.parametrize("size", [1e-17, 1e17])
def test_rows_near_both_ends_of_the_range(size, t, dtype):
    """silu(g) u near 2^-115 and 2^115, and slot weights of 1e-4."""
    w = layer(31, True)
    x = (torch.randn((t, D), generator=gen(35)) * size).to(DTYPES[dtype])
    idx, wts = choice(36, t)
    check(x, idx, wts * (1e-4 if size > 1 else 1.0), w, dtype, f"rows of {size}")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("t", [1, 40, 600])
def test_long_rows_whose_parts_differ_in_size(t, dtype):
    """f = 8448: 66 units of 128, the first two 2^-12 as large as the others and the last four 2^6 times, under down rows
    that take the units in part."""
    e, d, f = 4, 128, 8448
    w = [weight(51, (e,), f, d, 64, False), weight(52, (e,), f, d, 64, False), weight(53, (e,), d, f, 64, False)]
    for _, scales, _ in w[:2]:
        scales[:, :256] = (scales[:, :256].float() * 2.0 ** -6).half()
        scales[:, -512:] = (scales[:, -512:].float() * 2.0 ** 3).half()
    w[2][1][:, 64:] = (w[2][1][:, 64:].float() * 64).half()  # half of the outputs: the small units alone
    w[2][1][:, 64:, 4:] = 0
    x = torch.randn((t, d), generator=gen(55)).to(DTYPES[dtype])
    idx = torch.stack([torch.randperm(e, generator=gen(60 + i))[:K] for i in range(t)]).int()
    wts = torch.rand((t, K), generator=gen(56)) + 0.1
    note(f"[q4_moe long rows] T={t} {dtype}")
    y = bw.q4_moe(x.cuda(), idx.cuda(), wts.cuda(), *(bw.q4_upload(*(cuda(v) for v in m)) for m in w)).double()
    want = exact(x, idx, wts, w)
    for part in (slice(0, 64), slice(64, 128)):
        rel = float(((y - want)[:, part].norm(dim=1) / want[:, part].norm(dim=1)).max())
        note(f"  worst row {rel:.3g} (allowed {tolerance(dtype):.3g})")
        assert rel <= tolerance(dtype), part


@pytest.mark.parametrize("t", TOKENS)
def test_slot_weights_and_row_powers_do_not_underflow_together(t):
    """f32 rows whose silu(g) u lies near 2^-110, slot weights of 2^-14: the result is a normal number."""
    w = layer(41)
    x = torch.randn((t, D), generator=gen(45)) * 2.0 ** -54
    idx, wts = choice(46, t)
    check(x, idx, wts * 2.0 ** -14, w, "f32", "small rows and slot weights")
