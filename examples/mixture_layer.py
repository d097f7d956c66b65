"""A mixture-of-experts layer on 4-bit weights, and a few steps of tuning its router.

The layer, for hidden states x [T][d] (bfloat16):

    h      = x W_in^T                       q4_gemm
    logits = h W_router^T                   q4_gemm (32-bit activations: near ties decide experts)
    experts, weights = moe_route(logits)    sigmoid scores, balance bias, groups, renormalised
    y      = sum_j weights_j expert_j(h)    q4_moe
    out    = y W_out^T                      q4_gemm

The router is tuned through a vector b added to its logits, so that the weights of the chosen
experts come closer to given ones (moe_route_backward): loss = sum (weights - target)^2 / 2.

Run: python examples/mixture_layer.py [tokens]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_weight_gemm_amd as bw  # noqa: E402


def random_weight(gen, lead, n, k, group=128):
    """4-bit codes and scales of a weight whose products with unit rows are near 1: what a quantiser would give."""
    codes = torch.randint(0, 256, (*lead, n, k // 2), dtype=torch.uint8, device="cuda", generator=gen)
    scales = (0.5 + torch.rand((*lead, n, k // group), device="cuda", generator=gen)) * (0.2 / k ** 0.5)
    return codes, scales.half()


class MixtureLayer:
    def __init__(self, d=2048, f=1024, experts=64, chosen=8, groups=8, keep=4, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.chosen, self.groups, self.keep = chosen, groups, keep
        up = lambda *a: bw.q4_upload(*random_weight(gen, *a))  # noqa: E731
        self.w_in, self.w_out, self.router = up((), d, d), up((), d, d), up((), experts, d)
        self.gate, self.up, self.down = up((experts,), f, d), up((experts,), f, d), up((experts,), d, f)
        self.bias = 0.1 * torch.randn(experts, device="cuda", generator=gen)

    def logits(self, h):
        return bw.q4_gemm(self.router, h.float())

    def route(self, logits):
        return bw.moe_route(logits, self.chosen, bias=self.bias, score="sigmoid", groups=self.groups, keep=self.keep,
                            group_top=2, renorm=True)

    def __call__(self, x):
        h = bw.q4_gemm(self.w_in, x)
        idx, weights = self.route(self.logits(h))
        return bw.q4_gemm(self.w_out, bw.q4_moe(h, idx, weights, self.gate, self.up, self.down))


def tune(layer, h, target, steps, rate):
    """Losses of `steps` gradient steps on b; target(idx): the wanted weights [T][chosen]."""
    base = layer.logits(h)
    b, losses = torch.zeros(base.shape[1], device="cuda"), []
    idx, _ = layer.route(base)  # the choice stays; its weights move
    want = target(idx)
    for _ in range(steps):
        logits = base + b
        scores = torch.sigmoid(logits.gather(1, idx.long()))
        dw = scores / scores.sum(1, keepdim=True) - want
        losses.append(float((dw ** 2).sum() / 2))
        b -= rate * bw.moe_route_backward(logits, idx, dw, score="sigmoid", renorm=True).sum(0)
    return losses


def main():
    tokens = int(sys.argv[1]) if len(sys.argv) > 1 else 256
    layer = MixtureLayer()
    x = torch.randn((tokens, 2048), device="cuda").bfloat16()
    layer(x)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        layer(x)
    end.record()
    torch.cuda.synchronize()
    print(f"{tokens} tokens: {start.elapsed_time(end) / 20 * 1e3:.1f} us a pass")
    losses = tune(layer, bw.q4_gemm(layer.w_in, x), lambda idx: torch.full(idx.shape, 1 / 8, device="cuda"), 20, 0.5)
    print("router loss " + " ".join(f"{v:.4f}" for v in losses))


if __name__ == "__main__":
    main()
