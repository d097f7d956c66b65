"""Cases that measure the operators of a block around 4-bit weights.

Operators: `q4_linear` (product with a 4-bit weight, with bias, activation and residual in its epilogue), `moe_layer` (a whole
mixture-of-experts layer: norm, router, experts, residual), `block_norm` (the norms after and before a block, with its gate and
residual scale) and `block_norm_backward` (its gradient).

A 4-bit weight [N][K] is held as `codes` uint8 [N][K/2] (element 2j in the low four bits, 2j+1 in the high ones), `scales`
[N][K/G] for groups of G elements along K, and optionally `zeros` uint8 [N][K/G] (8 without them): W = (code - zero) * scale.

    q4_linear    y = act(x W^T + bias) + residual
    moe_layer    n = x / rms(x) * norm, rounded to x's type (n = x without a norm); logits = n R^T, summed in 64 bits and rounded to
                 32; experts and weights by the router's rule on those logits; y = residual + sum_j w_j down_j(silu(gate_j n) * up_j n)
    block_norm   u = norm(b) * post; y = x + scale * gate * u, rounded to x's type; n = norm(y) * pre
                 (norm: v / rms(v), or (v - mean(v)) / std(v) with a bias after its weight)
Where `own` is false, `run` is the plain form in elementary torch operations; where it is true, it calls this repository's operators.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6


def listed():
    return [
        # one token through an attention's output projection: bias and the residual stream
        dict(name="linear one row", op="linear", M=1, N=4096, K=4096, G=128, zeros=False, dtype="bf16", bias=True,
             act=None, residual=True),
        # a small batch of decoding requests through an MLP up-projection, fine groups with zero points
        dict(name="linear eight rows fine groups", op="linear", M=8, N=14336, K=4096, G=32, zeros=True, dtype="f16", bias=True,
             act="gelu_tanh", residual=False),
        # odd sizes, full-precision activations, a few rows
        dict(name="linear odd sizes f32", op="linear", M=23, N=5003, K=4000, G=32, zeros=True, dtype="f32", bias=True,
             act="silu", residual=True),
        # a prompt of 2048 tokens through a square projection with every part of the epilogue
        dict(name="linear prompt", op="linear", M=2048, N=4096, K=4096, G=128, zeros=False, dtype="bf16", bias=True,
             act="gelu", residual=True),
        # one decoding token through a whole layer, 8 of 64 experts
        dict(name="layer one token", op="layer", T=1, E=64, k=8, d=2048, f=1024, G=128, zeros=False, dtype="bf16",
             score="softmax", bias=False, groups=1, keep=1, group_top=1, renorm=True, norm=True, residual=True),
        # a small batch of decoding requests, sigmoid router with a balance bias and groups
        dict(name="layer eight tokens", op="layer", T=8, E=64, k=6, d=2048, f=1024, G=128, zeros=False, dtype="bf16",
             score="sigmoid", bias=True, groups=8, keep=4, group_top=2, renorm=True, norm=True, residual=True),
        # more requests over smaller experts, zero points, no norm of its own
        dict(name="layer batch", op="layer", T=33, E=32, k=4, d=1024, f=1536, G=64, zeros=True, dtype="f16",
             score="softmax", bias=False, groups=1, keep=1, group_top=1, renorm=False, norm=False, residual=True),
        # a short prompt in full precision through a few experts
        dict(name="layer short prompt f32", op="layer", T=200, E=8, k=2, d=1024, f=1024, G=128, zeros=False, dtype="f32",
             score="softmax", bias=False, groups=1, keep=1, group_top=1, renorm=True, norm=True, residual=False),
        # the norms between two blocks for one decoding token
        dict(name="norm one row", op="norm", M=1, N=4096, dtype="bf16", kind="rms", post=True, pre=True, rows=1, scale=1.0),
        # the same for a prompt of 4096 tokens
        dict(name="norm prompt", op="norm", M=4096, N=4096, dtype="bf16", kind="rms", post=True, pre=True, rows=1, scale=0.5),
        # its gradient in a training step, with a learned gate per channel
        dict(name="norm gradient", op="norm_backward", M=4096, N=4096, dtype="bf16", kind="rms", post=True, pre=True, rows=1,
             scale=0.5),
        # odd sizes, layer norms with biases, full precision, a gate for each of seven sequences
        dict(name="norm gradient odd f32", op="norm_backward", M=1001, N=1111, dtype="f32", kind="layer", post=True, pre=True,
             rows=7, scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "layer", "layer", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "f16", "f32"])
    G = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.5
    if op == "linear":
        N = _log(rng, 64, 14336)
        K = G * max(1, _log(rng, 256, 8192) // G)
        most = min(2048, (2048 * 4096 * 4096) // (N * K * (2 if dtype == "f32" else 1)))
        return dict(op=op, M=_log(rng, 1, most), N=N, K=K, G=G, zeros=zeros, dtype=dtype, bias=rng.random() < 0.7,
                    act=rng.choice([None, "relu", "gelu", "gelu_tanh", "silu"]), residual=rng.random() < 0.7)
    if op == "layer":
        groups = rng.choice([1, 1, 2, 4])
        E = groups * rng.randint(max(2, 4 // groups), 64 // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(8, keep * (E // groups)))
        d, f = G * max(1, _log(rng, 256, 2048) // G), G * max(1, _log(rng, 256, 1024) // G)
        return dict(op=op, T=_log(rng, 1, 256), E=E, k=k, d=d, f=f, G=G, zeros=zeros, dtype=dtype,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, keep=keep,
                    group_top=rng.choice([1, 2]) if groups > 1 else 1, renorm=rng.random() < 0.5, norm=rng.random() < 0.7,
                    residual=rng.random() < 0.7)
    N = _log(rng, 32, 8192)
    rows = rng.choice([1, 1, 4, 7])
    M = rows * max(1, _log(rng, 1, (4096 if dtype != "f32" else 2048)) // rows)
    post = rng.random() < 0.7
    return dict(op=op, M=M, N=N, dtype=dtype, kind=rng.choice(["rms", "layer"]), post=post, pre=rng.random() < 0.8 or not post,
                rows=rows, scale=rng.choice([1.0, 0.5, 0.22]))


# ---------------------------------------------------------------- inputs


def _weight(gen, lead, N, K, G, zeros):
    """Codes over all sixteen values, scales around 1/sqrt(5 K) (so that outputs are near 1)."""
    codes = torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = (0.5 + torch.rand((*lead, N, K // G), device="cuda", generator=gen)) * (0.2 / K ** 0.5)
    z = torch.randint(6, 11, (*lead, N, K // G), dtype=torch.uint8, device="cuda", generator=gen) if zeros else None
    return codes, s.half(), z


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    c, s, t = case, {}, DTYPES[case["dtype"]]

    def randn(*shape, about=0.0, width=1.0, dtype=t):
        return (about + width * torch.randn(shape, device="cuda", generator=gen)).to(dtype)

    if c["op"] == "linear":
        s["w"] = _weight(gen, (), c["N"], c["K"], c["G"], c["zeros"])
        s["x"] = randn(c["M"], c["K"])
        s["bias"] = randn(c["N"], width=0.5) if c["bias"] else None
        s["residual"] = randn(c["M"], c["N"], width=2.0) if c["residual"] else None
    elif c["op"] == "layer":
        for name, n, k in (("gate", c["f"], c["d"]), ("up", c["f"], c["d"]), ("down", c["d"], c["f"])):
            s[name] = _weight(gen, (c["E"],), n, k, c["G"], c["zeros"])
        # hidden states of a residual stream have a scale of their own; without a norm in the layer they come normed
        s["x"] = randn(c["T"], c["d"], width=3.0 if c["norm"] else 1.0)
        s["norm"] = randn(c["d"], about=1.0, width=0.1) if c["norm"] else None
        s["router"] = randn(c["E"], c["d"], width=c["d"] ** -0.5, dtype=torch.float32)
        s["bias"] = randn(c["E"], width=0.1, dtype=torch.float32) if c["bias"] else None
        s["residual"] = s["x"] if c["residual"] else None
    else:
        M, N = c["M"], c["N"]
        layer = c["kind"] == "layer"
        s["b"], s["x"] = randn(M, N), randn(M, N, about=0.2 if layer else 0.0, width=2.0)
        s["gate"] = randn(c["rows"], N, about=0.5, width=0.2)
        for name in ("post", "pre"):
            s[name] = randn(N, about=1.0, width=0.1) if c[name] else None
            s[name + "_bias"] = randn(N, width=0.1) if c[name] and layer else None
        if c["op"] == "norm_backward":
            s["dy"] = randn(M, N, width=0.01)
            s["dn"] = randn(M, N, width=0.01) if c["pre"] else None
            s["y"] = _plain_norm(dict(s, case=c))["y"]  # what the forward pass kept
    return s


def prepare(case, seed):
    """The inputs; for the operators also what a program keeps of its weights (uploaded once) and its output buffers."""
    s = dict(_inputs(case, seed), case=case)
    if own:
        import bit_weight_gemm_amd as bw

        s["bw"] = bw
        c, t = case, DTYPES[case["dtype"]]
        new = lambda *shape, dtype=t: torch.empty(shape, dtype=dtype, device="cuda")  # noqa: E731
        if c["op"] == "linear":
            s["w"] = bw.q4_upload(*s["w"])
            s["out"] = new(c["M"], c["N"])
        elif c["op"] == "layer":
            for name in ("gate", "up", "down"):
                s[name] = bw.q4_upload(*s[name])
            s["out"], s["idx"] = new(c["T"], c["d"]), new(c["T"], c["k"], dtype=torch.int32)
            s["weights"] = new(c["T"], c["k"], dtype=torch.float32)
        elif c["op"] == "norm":
            s["out"], s["n"] = new(c["M"], c["N"]), new(c["M"], c["N"]) if c["pre"] else None
    return s


# ---------------------------------------------------------------- plain forms (32 bits; 64 where ranks are decided)


def _dequant(w, t=torch.float32):
    codes, scales, zeros = w
    lead, K = codes.shape[:-1], 2 * codes.shape[-1]
    q = torch.stack((codes & 15, codes >> 4), -1).to(t).view(*lead, scales.shape[-1], -1)
    z = 8.0 if zeros is None else zeros.to(t)[..., None]
    return ((q - z) * scales.to(t)[..., None]).view(*lead, K)


def _plain_linear(s):
    z = s["x"].float() @ _dequant(s["w"]).T
    if s["bias"] is not None:
        z = z + s["bias"].float()
    act = s["case"]["act"]
    if act == "relu":
        z = torch.where(z > 0, z, torch.where(z != z, z, 0.0))
    elif act == "gelu":
        z = 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    elif act == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z))
    elif act == "silu":
        z = z * torch.sigmoid(z)
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(s["x"].dtype)


def _plain_route(c, logits, bias):
    l64 = logits.double()
    score = torch.softmax(l64, 1) if c["score"] == "softmax" else torch.sigmoid(l64)
    ranked = l64 if bias is None and c["group_top"] == 1 else score if bias is None else score + bias.double()
    if c["groups"] > 1:
        by_group = ranked.view(len(ranked), c["groups"], -1)
        best = by_group.topk(min(c["group_top"], by_group.shape[2]), 2).values.sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        ranked = torch.where(allowed[:, :, None], by_group, -math.inf).view(len(ranked), -1)
    idx = torch.sort(ranked, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    w = score.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, w.float()


def _plain_layer(s):
    c, rows = s["case"], s["x"]
    T, k, E = c["T"], c["k"], c["E"]
    if c["norm"]:  # in 64 bits: the rows' roundings decide experts too
        v = rows.double()
        rows = (v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * s["norm"].double()).to(rows.dtype)
    logits = (rows.double() @ s["router"].double().T).float()
    idx, w = _plain_route(c, logits, s["bias"])
    x = rows.float()
    if T * k <= E:  # few slots: each with its own expert's weights
        e = idx.flatten()
        gate, up, down = (_dequant(tuple(None if t is None else t[e] for t in s[n])) for n in ("gate", "up", "down"))
        each = x.repeat_interleave(k, 0)[:, None, :]
        g, u = torch.bmm(each, gate.transpose(1, 2)), torch.bmm(each, up.transpose(1, 2))
        out = torch.bmm(g * torch.sigmoid(g) * u, down.transpose(1, 2)).view(T, k, -1)
    else:  # the slots of each expert side by side, padded to the fullest expert
        e = idx.flatten()
        order = torch.sort(e, stable=True).indices
        count = torch.bincount(e, minlength=E)
        start = torch.cumsum(count, 0) - count
        most = int(count.max())
        place = torch.empty_like(e)
        place[order] = torch.arange(T * k, device=e.device) - start[e[order]]
        place = e * most + place
        each = torch.zeros((E * most, c["d"]), device=x.device)
        each[place] = x.repeat_interleave(k, 0)
        each = each.view(E, most, -1)
        g = torch.bmm(each, _dequant(s["gate"]).transpose(1, 2))
        h = g * torch.sigmoid(g) * torch.bmm(each, _dequant(s["up"]).transpose(1, 2))
        out = torch.bmm(h, _dequant(s["down"]).transpose(1, 2)).view(E * most, -1)[place].view(T, k, -1)
    y = (out * w[..., None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["x"].dtype), "idx": idx.int(), "weights": w}


def _hat(v, kind):
    """v normed, and what it was divided by."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    std = torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v / std, std


def _plain_norm(s):
    c, kind = s["case"], s["case"]["kind"]
    u = s["b"].float()
    if s["post"] is not None:
        u = _hat(u, kind)[0] * s["post"].float()
        if s["post_bias"] is not None:
            u = u + s["post_bias"].float()
    gate = s["gate"].float().repeat_interleave(c["M"] // c["rows"], 0)
    y = (s["x"].float() + c["scale"] * gate * u).to(s["x"].dtype)
    if s["pre"] is None:
        return {"y": y}
    n = _hat(y.float(), kind)[0] * s["pre"].float()
    if s["pre_bias"] is not None:
        n = n + s["pre_bias"].float()
    return {"y": y, "n": n.to(y.dtype)}


def _plain_norm_backward(s):
    c, kind = s["case"], s["case"]["kind"]

    def back(g, hat, std):
        """Gradient before a norm from the gradient after it."""
        g = g - hat * (g * hat).mean(1, keepdim=True) - (g.mean(1, keepdim=True) if kind == "layer" else 0.0)
        return g / std

    out, dx = {}, s["dy"].float()
    if s["pre"] is not None:
        hat, std = _hat(s["y"].float(), kind)
        dn = s["dn"].float()
        out["dpre"] = (dn * hat).sum(0)
        if s["pre_bias"] is not None:
            out["dpre_bias"] = dn.sum(0)
        dx = dx + back(dn * s["pre"].float(), hat, std)
    u, db = s["b"].float(), None
    du = c["scale"] * s["gate"].float().repeat_interleave(c["M"] // c["rows"], 0) * dx
    if s["post"] is not None:
        hat, std = _hat(u, kind)
        u = hat * s["post"].float()
        out["dpost"] = (du * hat).sum(0)
        if s["post_bias"] is not None:
            u = u + s["post_bias"].float()
            out["dpost_bias"] = du.sum(0)
        db = back(du * s["post"].float(), hat, std)
    else:
        db = du
    out["dgate"] = c["scale"] * (u * dx).view(c["rows"], -1, c["N"]).sum(1)
    t = s["dy"].dtype
    return dict(out, dx=dx.to(t), db=db.to(t))


PLAIN = {"linear": _plain_linear, "layer": _plain_layer, "norm": _plain_norm, "norm_backward": _plain_norm_backward}


def run(state):
    s, c = state, state["case"]
    if not own:
        return PLAIN[c["op"]](s)
    bw = s["bw"]
    if c["op"] == "linear":
        return bw.q4_linear(s["w"], s["x"], bias=s["bias"], activation=c["act"], residual=s["residual"], y=s["out"])
    if c["op"] == "layer":
        y, idx, w = bw.moe_layer(s["x"], s["router"], s["gate"], s["up"], s["down"], c["k"], norm=s["norm"], eps=EPS,
                                 bias=s["bias"], score=c["score"], groups=c["groups"], keep=c["keep"],
                                 group_top=c["group_top"], renorm=c["renorm"], residual=s["residual"], y=s["out"],
                                 idx=s["idx"], weights=s["weights"])
        return {"y": y, "idx": idx, "weights": w}
    if c["op"] == "norm":
        y, n = bw.block_norm(s["x"], b=s["b"], post=s["post"], post_bias=s["post_bias"], gate=s["gate"], scale=c["scale"],
                             pre=s["pre"], pre_bias=s["pre_bias"], kind=c["kind"], eps=EPS, y=s["out"], n=s["n"])
        return {"y": y} if n is None else {"y": y, "n": n}
    # names of its results: dx, db, dgate, and dpre, dpre_bias, dpost, dpost_bias where there are such parameters
    return bw.block_norm_backward(s["dy"], s["y"], dn=s["dn"], b=s["b"], post=s["post"], post_bias=s["post_bias"],
                                  gate=s["gate"], scale=c["scale"], pre=s["pre"], pre_bias=s["pre_bias"], kind=c["kind"],
                                  eps=EPS)


# ---------------------------------------------------------------- what a pass cannot do without


def _weight_bytes(N, K, G, zeros):
    return N * K // 2 + N * (K // G) * (3 if zeros else 2)


def work(case):
    c, b = case, SIZE[case["dtype"]]
    if c["op"] == "linear":
        return {"bytes": _weight_bytes(c["N"], c["K"], c["G"], c["zeros"]) + c["M"] * (c["K"] + c["N"]) * b +
                (c["N"] * b if c["bias"] else 0) + (c["M"] * c["N"] * b if c["residual"] else 0),
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "layer":
        touched = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"])  # experts that some token chose, if all are as likely
        one = 2 * _weight_bytes(c["f"], c["d"], c["G"], c["zeros"]) + _weight_bytes(c["d"], c["f"], c["G"], c["zeros"])
        return {"bytes": touched * one + 4 * c["E"] * c["d"] + 2 * c["T"] * c["d"] * b + 8 * c["T"] * c["k"],
                "flops": 6.0 * c["T"] * c["k"] * c["d"] * c["f"] + 2.0 * c["T"] * c["E"] * c["d"]}
    rows, par = c["M"] * c["N"] * b, c["N"] * b * (c["rows"] + (2 if c["kind"] == "layer" else 1) * (c["post"] + c["pre"]))
    if c["op"] == "norm":
        return {"bytes": (3 + c["pre"]) * rows + par, "flops": 12.0 * c["M"] * c["N"]}
    # dy, b, dx, db, and with a norm behind the sum y and dn
    return {"bytes": (4 + 2 * c["pre"]) * rows + par + par // b * 4, "flops": 30.0 * c["M"] * c["N"]}


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


def _exact_linear(s):
    z = s["x"].double() @ _w64(s["w"]).T.contiguous()
    if s["bias"] is not None:
        z += s["bias"].double()[None]
    act = s["case"]["act"]
    if act == "relu":
        z = z.clamp(min=0.0)
    elif act == "gelu":
        z = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
    elif act == "gelu_tanh":
        z = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    elif act == "silu":
        z = z / (1.0 + torch.exp(-z))
    return z if s["residual"] is None else z + s["residual"].double()


def _place(v):
    """How many entries of its row come before each: larger ones, and equal ones of lower index."""
    before = torch.ones((v.shape[1],) * 2, dtype=torch.bool, device=v.device).tril(-1)
    return ((v[:, None, :] > v[:, :, None]) | ((v[:, None, :] == v[:, :, None]) & before)).sum(2)


def _exact_layer(s):
    c, t = s["case"], s["x"].dtype
    n = s["x"].double()
    if c["norm"]:
        n = (n / (n.pow(2).sum(1, keepdim=True) / c["d"] + EPS).sqrt() * s["norm"].double()).to(t).double()
    l = torch.stack([(n * row).sum(1) for row in s["router"].double()], 1).float().double()
    p = torch.exp(l - l.max(1, keepdim=True).values)
    p = p / p.sum(1, keepdim=True) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-l))
    key = p + s["bias"].double() if s["bias"] is not None else (l if c["group_top"] == 1 else p)
    m = c["E"] // c["groups"]
    if c["groups"] > 1:
        best = key.view(c["T"], c["groups"], m).sort(2, descending=True).values[:, :, : c["group_top"]].sum(2)
        key = torch.where(_place(best).repeat_interleave(m, 1) < c["keep"], key, -math.inf)
    place = _place(key)
    idx = torch.stack([(place == j).int().argmax(1) for j in range(c["k"])], 1)
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    y = torch.zeros((c["T"], c["d"]), dtype=torch.float64, device=n.device)
    for e in range(c["E"]):
        row, j = (idx == e).nonzero(as_tuple=True)
        if len(row):
            part = lambda name: _w64(tuple(None if v is None else v[e] for v in s[name])).T.contiguous()  # noqa: E731
            g, u = n[row] @ part("gate"), n[row] @ part("up")
            y.index_add_(0, row, (g / (1 + torch.exp(-g)) * u) @ part("down") * w[row, j][:, None])
    if s["residual"] is not None:
        y += s["residual"].double()
    return {"y": y, "idx": idx.int(), "weights": w}


def _normed64(v, kind, weight, bias):
    """norm(v) * weight + bias."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v / (v.pow(2).mean(1, keepdim=True) + EPS).sqrt() * weight
    return v if bias is None else v + bias


def _wide(s, *names):
    return [None if s[name] is None else s[name].double() for name in names]


def _exact_norm(s):
    c = s["case"]
    b, x, gate, post, post_bias, pre, pre_bias = _wide(s, "b", "x", "gate", "post", "post_bias", "pre", "pre_bias")
    u = b if post is None else _normed64(b, c["kind"], post, post_bias)
    y = (x.view(c["rows"], -1, c["N"]) + c["scale"] * gate[:, None, :] * u.view(c["rows"], -1, c["N"])).view(x.shape)
    return {"y": y} if pre is None else {"y": y, "n": _normed64(y.to(s["x"].dtype).double(), c["kind"], pre, pre_bias)}


def _exact_norm_backward(s):
    """By autograd in 64 bits: the loss dy . y + dn . n, with n a function of y."""
    c = s["case"]
    with torch.enable_grad():
        leaf = {name: s[name].double().requires_grad_() for name in ("b", "gate", "post", "post_bias", "pre", "pre_bias")
                if s[name] is not None}
        get = leaf.get
        total = s["dy"].double()
        if "pre" in leaf:
            y = s["y"].double().requires_grad_()
            (_normed64(y, c["kind"], get("pre"), get("pre_bias")) * s["dn"].double()).sum().backward()
            total = total + y.grad
        u = leaf["b"] if "post" not in leaf else _normed64(leaf["b"], c["kind"], get("post"), get("post_bias"))
        shape = (c["rows"], -1, c["N"])
        (c["scale"] * leaf["gate"][:, None, :] * u.view(shape) * total.view(shape)).sum().backward()
    return dict({"d" + name: v.grad for name, v in leaf.items()}, dx=total)


def exact(case, seed):
    s = dict(_inputs(case, seed), case=case)
    return {"linear": _exact_linear, "layer": _exact_layer, "norm": _exact_norm, "norm_backward": _exact_norm_backward}[case["op"]](s)
