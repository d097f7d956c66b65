"""References in 64 bits and argument structs of the tests of a block's operators (test infrastructure)."""

import ctypes
import math

import torch

from q4_util import DTYPES, dequant64, moe64, route64

P, I64, I32, F64, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_float
CODES = {"f32": 0, "f16": 1, "bf16": 2}


class LayerCall(ctypes.Structure):
    _fields_ = [(n, P) for n in ("x", "norm", "router", "bias", "gate", "up", "down", "residual", "y", "idx", "weights")] + \
               [("eps", F64)] + [(n, I64) for n in ("T", "k", "groups", "keep", "group_top")] + \
               [(n, I32) for n in ("score", "renorm", "dtype", "norm_dtype", "router_dtype", "reserved")]


class NormCall(ctypes.Structure):
    _fields_ = [(n, P) for n in ("x", "b", "post", "post_bias", "gate", "pre", "pre_bias", "y", "n")] + [("eps", F64)] + \
               [(n, I64) for n in ("M", "N", "R")] + [("scale", F32)] + [(n, I32) for n in ("layer", "dtype", "weights_dtype")]


class NormBackwardCall(ctypes.Structure):
    _fields_ = [(n, P) for n in ("dy", "dn", "y", "b", "post", "post_bias", "gate", "pre", "pre_bias", "dx", "db", "dgate", "dpost",
                                 "dpost_bias", "dpre", "dpre_bias")] + [("eps", F64)] + \
               [(n, I64) for n in ("M", "N", "R")] + [("scale", F32)] + [(n, I32) for n in ("layer", "dtype", "weights_dtype")]


def half_step(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def least(dtype):
    """Half a step of the type's subnormal numbers."""
    return {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}[dtype]


def act64(name, z):
    if name is None:
        return z
    if name == "relu":
        return torch.where(z < 0, 0.0, z)
    low = z == -math.inf
    if name == "gelu":
        out = z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    elif name == "gelu_tanh":
        out = 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    else:
        out = z / (1.0 + torch.exp(-z))
    return torch.where(low, 0.0, out)


def hat64(v, kind, eps):
    """v normed, in f64."""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v / ((v * v).mean(1, keepdim=True) + eps).sqrt()


def norm64(v, kind, eps, weight, bias):
    v = hat64(v, kind, eps) * weight
    return v if bias is None else v + bias


def u64(b, post, post_bias, kind, eps):
    return b if post is None else norm64(b, kind, eps, post, post_bias)


def d64(t):
    return None if t is None else t.double()


def layer64(x, router, gate, up, down, k, norm=None, eps=1e-6, bias=None, score="softmax", groups=1, keep=1, group_top=1,
            renorm=False, residual=None):
    """The layer from its definition on the CPU: (moe part f64, idx, weights f64, logits f32)."""
    n = x
    if norm is not None:
        v = x.double()
        n = (v / ((v * v).mean(1, keepdim=True) + eps).sqrt() * norm.double()).to(x.dtype)
    logits = (n.double() @ router.double().T).float()
    idx, w = route64(logits, k, bias, score, groups, keep, group_top, renorm)
    return moe64(n, idx, w, *(dequant64(*v) for v in (gate, up, down))), idx, w, logits
