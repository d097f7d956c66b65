"""Inputs and 64-bit references of the 4-bit weight and mixture-of-experts tests (test infrastructure)."""

import math

import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def weight(seed, lead, n, k, group, zeros, scale=None):
    """codes, scales, zeros on the CPU; every code and, with zeros, zero points 0 .. 15."""
    g = gen(seed)
    codes = torch.randint(0, 256, (*lead, n, k // 2), dtype=torch.uint8, generator=g)
    scale = 0.2 / math.sqrt(k) if scale is None else scale
    scales = ((0.5 + torch.rand((*lead, n, k // group), generator=g)) * scale).half()
    z = torch.randint(0, 16, (*lead, n, k // group), dtype=torch.uint8, generator=g) if zeros else None
    return codes, scales, z


def dequant64(codes, scales, zeros):
    """(code - zero) * scale in f64, element by element from the format's definition."""
    k = 2 * codes.shape[-1]
    q = torch.empty((*codes.shape[:-1], k), dtype=torch.float64)
    q[..., 0::2] = (codes & 15).double()
    q[..., 1::2] = (codes >> 4).double()
    group = k // scales.shape[-1]
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(group, -1)
    return (q - z) * scales.double().repeat_interleave(group, -1)


def cuda(t):
    return None if t is None else t.cuda()


def route64(logits, k, bias, score, groups, keep, group_top, renorm):
    """The router from its definition, row by row on the CPU: (idx, weights) in f64."""
    t, e = logits.shape
    n = e // groups
    idx = torch.full((t, k), -1, dtype=torch.int32)
    out = torch.zeros((t, k), dtype=torch.float64)
    for row in range(t):
        l = logits[row].double()
        masked = l == -math.inf
        if score == "sigmoid":
            p = 1.0 / (1.0 + torch.exp(-l))
        elif masked.all():
            p = torch.zeros_like(l)
        else:
            p = torch.exp(l - l.max())
            p = p / p.sum()
        key = (p + bias.double()) if bias is not None else (l.clone() if group_top == 1 or groups == 1 else p.clone())
        key[masked] = -math.inf
        key = torch.where(key.isnan(), math.inf, key).tolist()
        if groups > 1:
            best = []
            for g in range(groups):
                v = sorted(key[g * n: (g + 1) * n], reverse=True)[:group_top]
                v = v[:1] + [a for a in v[1:] if a != -math.inf]
                best.append(sum(v))
            kept = sorted(range(groups), key=lambda g: (-best[g], g))[:keep]
            key = [v if i // n in kept else -math.inf for i, v in enumerate(key)]
        order = [i for i in sorted(range(e), key=lambda i: (-key[i], i)) if key[i] != -math.inf][:k]
        idx[row, : len(order)] = torch.tensor(order, dtype=torch.int32)
        out[row, : len(order)] = p[order]
        total = out[row].sum()
        if renorm and total != 0:
            out[row] /= total
    return idx, out


def route_weights64(logits, idx, score, renorm):
    """The chosen weights as a differentiable f64 function of the logits, the choice held fixed."""
    p = torch.softmax(logits, 1) if score == "softmax" else 1.0 / (1.0 + torch.exp(-logits))
    on = (idx >= 0) & (idx < logits.shape[1])
    c = torch.where(on, p.gather(1, idx.long().clamp(0, logits.shape[1] - 1)), 0.0)
    return c / c.sum(1, keepdim=True) if renorm else c


def moe64(x, idx, weights, gate, up, down):
    """Token by token, slot by slot, in f64; gate, up, down: dequantised [E][..][..] f64."""
    y = torch.zeros((x.shape[0], down.shape[1]), dtype=torch.float64)
    e_all = gate.shape[0]
    for t in range(x.shape[0]):
        xt = x[t].double()
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if 0 <= e < e_all:
                g, u = gate[e] @ xt, up[e] @ xt
                y[t] += weights[t, j].double() * (down[e] @ (g / (1.0 + torch.exp(-g)) * u))
    return y
