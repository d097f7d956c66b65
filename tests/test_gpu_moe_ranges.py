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


@pytest.mark.parametrize("t", TOKENS)
def test_slot_weights_and_row_powers_do_not_underflow_together(t):
    """f32 rows whose silu(g) u lies near 2^-110, slot weights of 2^-14: the result is a normal number."""
    w = layer(41)
    x = torch.randn((t, D), generator=gen(45)) * 2.0 ** -54
    idx, wts = choice(46, t)
    check(x, idx, wts * 2.0 ** -14, w, "f32", "small rows and slot weights")
