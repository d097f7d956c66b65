"""Cases that measure the 4-bit weight product and the mixture-of-experts operators.

Operators: `q4_gemm` (product with a 4-bit weight under group scales), `moe_route`
(router scores to chosen experts and their weights), `moe_route_backward` (its gradient)
and `q4_moe` (the chosen experts' gated products over 4-bit weights, summed per token).

A 4-bit weight [N][K] is held as `codes` uint8 [N][K/2] (element 2j in the low four bits,
2j+1 in the high ones), `scales` [N][K/G] for groups of G elements along K, and optionally
`zeros` uint8 [N][K/G] (8 without them): W = (code - zero) * scale.  Experts are stacked
along a leading axis.  Where `own` is false, `run` is the plain form in elementary torch
operations; where it is true, it calls this repository's operators.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


def listed():
    return [
        # one token through a square projection: the decode step of a dense layer
        dict(name="q4 one row", op="gemm", M=1, N=4096, K=4096, G=128, zeros=False, dtype="bf16"),
        # a small batch of decoding requests through an MLP up-projection, fine groups with zero points
        dict(name="q4 eight rows fine groups", op="gemm", M=8, N=14336, K=4096, G=32, zeros=True, dtype="f16"),
        # odd sizes, full-precision activations, a few rows
        dict(name="q4 odd sizes f32", op="gemm", M=23, N=5003, K=4000, G=32, zeros=True, dtype="f32"),
        # a prompt of 2048 tokens through the same square projection
        dict(name="q4 prompt", op="gemm", M=2048, N=4096, K=4096, G=128, zeros=False, dtype="bf16"),
        # one token's router: sigmoid scores, a balance bias, 4 of 8 groups, renormalised weights
        dict(name="route one token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             group_top=2, renorm=True, dtype="f32"),
        # the same router over a long prompt
        dict(name="route prompt", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             group_top=2, renorm=True, dtype="f32"),
        # a softmax router without groups, logits in bf16 (equal logits are common there)
        dict(name="route softmax bf16", op="route", T=4096, E=64, k=6, score="softmax", bias=False, groups=1, keep=1,
             group_top=1, renorm=False, dtype="bf16"),
        # the router's gradient in a training step: dense softmax, and renormalised sigmoid
        dict(name="route gradient softmax", op="route_backward", T=8192, E=128, k=8, score="softmax", renorm=False,
             dtype="f32"),
        dict(name="route gradient sigmoid", op="route_backward", T=1000, E=64, k=6, score="sigmoid", renorm=True,
             dtype="bf16"),
        # one decoding token through 8 of 64 experts
        dict(name="experts one token", op="moe", T=1, E=64, k=8, d=2048, f=1024, G=128, zeros=False, dtype="bf16",
             drop=0.0),
        # a batch of decoding requests, zero points, some slots dropped
        dict(name="experts batch", op="moe", T=33, E=32, k=4, d=1024, f=1536, G=64, zeros=True, dtype="f16", drop=0.1),
        # a prompt of 2048 tokens through the 64 experts
        dict(name="experts prompt", op="moe", T=2048, E=64, k=8, d=2048, f=1024, G=128, zeros=False, dtype="bf16",
             drop=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _route_sizes(rng, T):
    groups = rng.choice([1, 1, 2, 4, 8])
    E = groups * rng.randint(max(2, 8 // groups), 256 // groups)
    keep = rng.randint(1, groups)
    k = rng.randint(1, min(8, keep * (E // groups)))
    return dict(T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                keep=keep, group_top=rng.choice([1, 2]) if groups > 1 else 1, renorm=rng.random() < 0.5)


def draw(rng):
    op = rng.choice(["gemm", "gemm", "route", "route_backward", "moe", "moe"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    G = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.5
    if op == "gemm":
        N = _log(rng, 64, 14336)
        K = G * max(1, _log(rng, 256, 8192) // G)
        most = min(2048, (2048 * 4096 * 4096) // (N * K * (2 if dtype == "f32" else 1)))
        return dict(op=op, M=_log(rng, 1, most), N=N, K=K, G=G, zeros=zeros, dtype=dtype)
    if op == "route":
        return dict(op=op, dtype=dtype, **_route_sizes(rng, _log(rng, 1, 16384)))
    if op == "route_backward":
        E = rng.randint(8, 256)
        return dict(op=op, T=_log(rng, 1, 4096), E=E, k=rng.randint(1, 8), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, dtype=dtype)
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    d, f = G * max(1, _log(rng, 256, 2048) // G), G * max(1, _log(rng, 256, 1024) // G)
    T = _log(rng, 1, 1024 if dtype == "f32" else 2048)
    return dict(op=op, T=T, E=E, k=k, d=d, f=f, G=G, zeros=zeros, dtype=dtype, drop=rng.choice([0.0, 0.1]))


# ---------------------------------------------------------------- inputs


def _weight(gen, lead, N, K, G, zeros):
    """Codes over all sixteen values, scales around 1/sqrt(5 K) (so that outputs are near 1)."""
    codes = torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (0.5 + torch.rand((*lead, N, K // G), device="cuda", generator=gen)) * (0.2 / K ** 0.5)
    z = torch.randint(6, 11, (*lead, N, K // G), dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return codes, s.half(), z


def _randn(gen, shape, dtype):
    return torch.randn(shape, device="cuda", generator=gen).to(DTYPES[dtype])


def _choice(gen, T, E, k, drop):
    """k distinct experts per token, some experts asked for more than others; dropped slots are -1."""
    pop = torch.randn(E, device="cuda", generator=gen)
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=gen).clamp(1e-9, 1 - 1e-6)))
    idx = torch.topk(pop + noise, k, dim=1).indices.int()
    if drop:
        idx = torch.where(torch.rand((T, k), device="cuda", generator=gen) < drop, -1, idx)
    w = torch.rand((T, k), device="cuda", generator=gen) + 0.1
    return idx.int().contiguous(), (w / w.sum(1, keepdim=True)).contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c, s = case, {}
    if c["op"] == "gemm":
        s["w"] = _weight(gen, (), c["N"], c["K"], c["G"], c["zeros"])
        s["x"] = _randn(gen, (c["M"], c["K"]), c["dtype"])
    elif c["op"] == "route":
        s["logits"] = _randn(gen, (c["T"], c["E"]), c["dtype"])
        s["bias"] = 0.1 * torch.randn(c["E"], device="cuda", generator=gen) if c["bias"] else None
    elif c["op"] == "route_backward":
        s["logits"] = _randn(gen, (c["T"], c["E"]), c["dtype"])
        s["idx"] = torch.topk(s["logits"].float(), c["k"], dim=1).indices.int().contiguous()
        s["dw"] = torch.randn((c["T"], c["k"]), device="cuda", generator=gen)
    else:
        for name, n, k in (("gate", c["f"], c["d"]), ("up", c["f"], c["d"]), ("down", c["d"], c["f"])):
            s[name] = _weight(gen, (c["E"],), n, k, c["G"], c["zeros"])
        s["x"] = _randn(gen, (c["T"], c["d"]), c["dtype"])
        s["idx"], s["weights"] = _choice(gen, c["T"], c["E"], c["k"], c["drop"])
    return s


def prepare(case, seed):
    """The inputs; for the operators also what a program keeps of its weights (uploaded once) and its output buffers."""
    s = dict(_inputs(case, seed), case=case)
    if own:
        import bit_weight_gemm_amd as bw

        s["bw"] = bw
        c = case
        if c["op"] == "gemm":
            s["w"] = bw.q4_upload(*s["w"])
            s["y"] = torch.empty((c["M"], c["N"]), dtype=DTYPES[c["dtype"]], device="cuda")
        elif c["op"] == "moe":
            for name in ("gate", "up", "down"):
                s[name] = bw.q4_upload(*s[name])
            s["y"] = torch.empty((c["T"], c["d"]), dtype=DTYPES[c["dtype"]], device="cuda")
        elif c["op"] == "route":
            s["idx"] = torch.empty((c["T"], c["k"]), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((c["T"], c["k"]), device="cuda")
        else:
            s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits; 64 where ranks are decided)


def _dequant(w, t=torch.float32):
    codes, scales, zeros = w
    lead, K = codes.shape[:-1], 2 * codes.shape[-1]
    q = torch.stack((codes & 15, codes >> 4), -1).to(t).view(*lead, scales.shape[-1], -1)
    z = 8.0 if zeros is None else zeros.to(t)[..., None]
    return ((q - z) * scales.to(t)[..., None]).view(*lead, K)


def _plain_gemm(s):
    return (s["x"].float() @ _dequant(s["w"]).T).to(s["x"].dtype)


def _plain_route(s):
    c, l64 = s["case"], s["logits"].double()
    score = torch.softmax(l64, 1) if c["score"] == "softmax" else torch.sigmoid(l64)
    ranked = l64 if s["bias"] is None and c["group_top"] == 1 else score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        by_group = ranked.view(c["T"], c["groups"], -1)
        best = by_group.topk(min(c["group_top"], by_group.shape[2]), 2).values.sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        ranked = torch.where(allowed[:, :, None], by_group, -math.inf).view(c["T"], -1)
    idx = torch.sort(ranked, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.int(), "weights": w.float()}


def _plain_route_backward(s):
    c, l, dw = s["case"], s["logits"].float(), s["dw"]
    idx = s["idx"].long()
    p = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
    chosen = p.gather(1, idx)
    if c["renorm"]:
        total = chosen.sum(1, keepdim=True)
        dchosen = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total
    else:
        dchosen = dw
    dp = torch.zeros_like(l).scatter(1, idx, dchosen)
    if c["score"] == "softmax":
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    else:
        dl = dp * p * (1 - p)
    return dl.to(s["logits"].dtype)


def _plain_moe(s):
    c, x, idx = s["case"], s["x"].float(), s["idx"].long()
    T, k, E = c["T"], c["k"], c["E"]
    if T * k <= E:  # few slots: each with its own expert's weights
        e = idx.clamp(min=0).flatten()
        gate, up, down = (_dequant(tuple(None if t is None else t[e] for t in s[n])) for n in ("gate", "up", "down"))
        rows = x.repeat_interleave(k, 0)[:, None, :]
        g, u = torch.bmm(rows, gate.transpose(1, 2)), torch.bmm(rows, up.transpose(1, 2))
        out = torch.bmm(g * torch.sigmoid(g) * u, down.transpose(1, 2)).view(T, k, -1)
    else:  # the slots of each expert side by side, padded to the fullest expert
        e = torch.where(idx < 0, E, idx).flatten()
        order = torch.sort(e, stable=True).indices
        count = torch.bincount(e, minlength=E + 1)
        start = torch.cumsum(count, 0) - count
        most = int(count[:E].max())
        place = torch.empty_like(e)
        place[order] = torch.arange(T * k, device=e.device) - start[e[order]]
        place = torch.where(e < E, e * most + place, E * most)  # one row past the end for dropped slots
        rows = torch.zeros((E * most + 1, c["d"]), device=x.device)
        rows[place] = x.repeat_interleave(k, 0)
        rows = rows[:-1].view(E, most, -1)
        g = torch.bmm(rows, _dequant(s["gate"]).transpose(1, 2))
        h = g * torch.sigmoid(g) * torch.bmm(rows, _dequant(s["up"]).transpose(1, 2))
        out = torch.bmm(h, _dequant(s["down"]).transpose(1, 2)).view(E * most, -1)
        out = torch.cat((out, out.new_zeros(1, c["d"])))[place].view(T, k, -1)
    w = torch.where(idx < 0, 0.0, s["weights"])
    return (out * w[..., None]).sum(1).to(s["x"].dtype)


PLAIN = {"gemm": _plain_gemm, "route": _plain_route, "route_backward": _plain_route_backward, "moe": _plain_moe}


def run(state):
    c = state["case"]
    if not own:
        return PLAIN[c["op"]](state)
    bw = state["bw"]
    if c["op"] == "gemm":
        return bw.q4_gemm(state["w"], state["x"], state["y"])
    if c["op"] == "moe":
        return bw.q4_moe(state["x"], state["idx"], state["weights"], state["gate"], state["up"], state["down"],
                         state["y"])
    if c["op"] == "route":
        idx, weights = bw.moe_route(state["logits"], c["k"], bias=state["bias"], score=c["score"], groups=c["groups"],
                                    keep=c["keep"], group_top=c["group_top"], renorm=c["renorm"], idx=state["idx"],
                                    weights=state["weights"])
        return {"idx": idx, "weights": weights}
    return bw.moe_route_backward(state["logits"], state["idx"], state["dw"], score=c["score"], renorm=c["renorm"],
                                 dlogits=state["dlogits"])


# ---------------------------------------------------------------- what a pass cannot do without


def _weight_bytes(N, K, G, zeros):
    return N * K // 2 + N * (K // G) * (3 if zeros else 2)


def work(case):
    c, b = case, SIZE[case["dtype"]]
    if c["op"] == "gemm":
        return {"bytes": _weight_bytes(c["N"], c["K"], c["G"], c["zeros"]) + c["M"] * (c["K"] + c["N"]) * b,
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * b + c["k"] * 8) + (4 * c["E"] if c["bias"] else 0),
                "flops": 8.0 * c["T"] * c["E"]}
    if c["op"] == "route_backward":
        return {"bytes": c["T"] * (2 * c["E"] * b + c["k"] * 8), "flops": 8.0 * c["T"] * c["E"]}
    touched = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts that some token chose, if all are as likely
    one = 2 * _weight_bytes(c["f"], c["d"], c["G"], c["zeros"]) + _weight_bytes(c["d"], c["f"], c["G"], c["zeros"])
    return {"bytes": touched * one + 2 * c["T"] * c["d"] * b + 8 * c["T"] * c["k"],
            "flops": 6.0 * c["T"] * c["k"] * (1 - c["drop"]) * c["d"] * c["f"]}


# ---------------------------------------------------------------- the definitions in 64 bits


def _w64(w):
    codes, scales, zeros = w
    K = 2 * codes.shape[-1]
    q = torch.empty((*codes.shape[:-1], K), dtype=torch.float64, device=codes.device)
    q[..., 0::2] = (codes % 16).double()
    q[..., 1::2] = (codes // 16).double()
    G = K // scales.shape[-1]
    q -= 8.0 if zeros is None else zeros.double().repeat_interleave(G, -1)
    return q * scales.double().repeat_interleave(G, -1)


def _exact_route(s):
    """Token by token in Python numbers for few tokens; the ranks are not repeated for many (None)."""
    c = s["case"]
    l = s["logits"].double()
    p = torch.exp(l - l.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    key = p + s["bias"].double() if s["bias"] is not None else (l if c["group_top"] == 1 else p)
    n = c["E"] // c["groups"]
    if c["groups"] > 1:
        # a group's place is the number of groups that beat it (equal ones: the lower index first)
        best = key.view(c["T"], c["groups"], n).sort(2, descending=True).values[:, :, : c["group_top"]].sum(2)
        key = torch.where(_place(best).repeat_interleave(n, 1) < c["keep"], key, -math.inf)
    # an expert's place likewise; the expert at place j goes to slot j
    place, idx = _place(key), torch.empty((c["T"], c["k"]), dtype=torch.int64, device=l.device)
    for j in range(c["k"]):
        idx[:, j] = (place == j).int().argmax(1)
    w = torch.gather(p, 1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.int(), "weights": w}


def _place(v):
    """How many entries of its row come before each: larger ones, and equal ones of lower index."""
    out = torch.empty(v.shape, dtype=torch.int32, device=v.device)
    before = torch.ones((v.shape[1],) * 2, dtype=torch.bool, device=v.device).tril(-1)
    for a in range(0, v.shape[0], 256):
        b = v[a: a + 256]
        out[a: a + 256] = ((b[:, None, :] > b[:, :, None]) | ((b[:, None, :] == b[:, :, None]) & before)).sum(2)
    return out


def _exact_route_backward(s):
    """By the Jacobian of the chosen weights, summed over the slots."""
    c, l, idx = s["case"], s["logits"].double(), s["idx"].long()
    p = torch.softmax(l, 1) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    ch, dw = p.gather(1, idx), s["dw"].double()
    out = torch.zeros_like(l)
    for j in range(c["k"]):
        for i in range(c["k"]) if c["renorm"] else (j,):
            # d w_j / d p_i, times dw_j
            a = (float(i == j) / ch.sum(1) - ch[:, j] / ch.sum(1) ** 2) if c["renorm"] else torch.ones_like(ch[:, 0])
            a = (a * dw[:, j])[:, None]
            pi, at = ch[:, i: i + 1], idx[:, i: i + 1]
            if c["score"] == "softmax":
                out -= a * pi * p
                out.scatter_add_(1, at, a * pi)
            else:
                out.scatter_add_(1, at, a * pi * (1 - pi))
    return out


def _exact_moe(s):
    c, x = s["case"], s["x"].double()
    out = torch.zeros((c["T"], c["d"]), dtype=torch.float64, device=x.device)
    for e in range(c["E"]):
        t, j = (s["idx"] == e).nonzero(as_tuple=True)
        if len(t):
            part = lambda n: _w64(tuple(None if v is None else v[e] for v in s[n]))  # noqa: E731
            g, u = x[t] @ part("gate").T.contiguous(), x[t] @ part("up").T.contiguous()
            o = (g / (1 + torch.exp(-g)) * u) @ part("down").T.contiguous()
            out.index_add_(0, t, o * s["weights"][t, j].double()[:, None])
    return out


def exact(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"] == "gemm":
        return s["x"].double() @ _w64(s["w"]).T.contiguous()
    return {"route": _exact_route, "route_backward": _exact_route_backward, "moe": _exact_moe}[case["op"]](s)
