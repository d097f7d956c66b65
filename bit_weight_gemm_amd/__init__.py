"""Python binding of libtq2 (ctypes): argument marshalling only.

Every step of the computation runs in the HIP kernels of libtq2.so; torch only
supplies device memory (tensors on the current GPU) and the current stream.
There is no CPU fallback: if the library is missing or fails to load, the calls
raise.

Names follow the C ABI in include/libtq2.h: tq2_upload, tq2_free, tq2_gemm,
tq2_gemm_path, tq2_dequant, blr_forward, blr_forward_paths, blr_backward_paths
(library-owned workspace), blr_forward_ws, blr_forward_paths_ws,
blr_backward_paths_ws (caller-owned workspace), blr_forward_paths_save and
blr_backward_paths_saved (activations kept by the forward for the backward),
blr_saved_size, blr_workspace_size,
blr_backward_workspace_size, tq2_workspace_allocs, tq2_select_path,
tq2_set_path, tq2_set_m_small, tq2_strerror, tq2_version; and in include/libtq2_moe.h:
q4_upload (packs into memory of its own), q4_gemm, q4_dequant, moe_route,
moe_route_backward and q4_moe.  The last three and q4_gemm go through a compiled
module (csrc/binding.cpp): beside their kernels' few microseconds, checks and
conversions in Python would be the larger part.

No call records anything for autograd: gradients come from the backward calls.

Every tensor's shape is checked here against the sizes the call derives from x,
h and l before anything reaches the library: the C ABI takes raw device
pointers and cannot see buffer sizes.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq2.so")

TQ2_OK, TQ2_EINVAL, TQ2_ENOMEM, TQ2_EDEVICE, TQ2_ENODEV, TQ2_ETOOBIG = 0, -1, -2, -3, -4, -5
TQ2_STATIC_SCRATCH_BYTES = 16 << 20
TQ2_PATH_AUTO, TQ2_PATH_F32, TQ2_PATH_MFMA = 0, 1, 2

_lib = None


class Tq2Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {tq2_strerror(status)} ({status})")


def _single_hip_runtime():
    """Fail if two different HIP runtimes are mapped (device pointers would not mix)."""
    try:
        with open("/proc/self/maps") as f:
            paths = {ln.split()[-1] for ln in f if "libamdhip64" in ln}
    except OSError:
        return
    real = {os.path.realpath(p) for p in paths}
    if len(real) > 1:
        raise RuntimeError(f"more than one HIP runtime loaded: {sorted(real)}")


def lib():
    """Load libtq2.so (after torch, so both share torch's HIP runtime)."""
    global _lib, _compiled
    if _lib is not None:
        return _lib
    import torch  # load torch's HIP runtime first

    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run bit_weight_gemm_amd/build.py")
    L = ctypes.CDLL(LIB_PATH)
    _single_hip_runtime()
    i64, sz, p, i32 = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int
    sig = {
        "tq2_upload": ([p, sz, i64, i64, p, ctypes.POINTER(p)], i32),
        "tq2_free": ([p], i32),
        "tq2_weight_info": ([p, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(sz)], i32),
        "tq2_gemm": ([p, p, p, i64, i64, i64, p], i32),
        "tq2_gemm_path": ([p, p, p, i64, i64, i64, i32, p], i32),
        "tq2_select_path": ([i64], i32),
        "tq2_set_m_small": ([i64], i64),
        "tq2_dequant": ([p, p, p], i32),
        "tq2_set_path": ([i32], i32),
        "tq2_workspace_allocs": ([], ctypes.c_uint64),
        "blr_workspace_size": ([i64, i64, i64, i64], sz),
        "blr_forward": ([p, p, p, p, p, p, p, i64, i64, i64, i64, p], i32),
        "blr_forward_paths": ([i64, p, p, p, p, p, p, p, i64, i64, i64, i64, p], i32),
        "blr_forward_noalloc": ([p, p, p, p, p, p, p, i64, i64, i64, i64, p], i32),
        "blr_forward_ws": ([p, p, p, p, p, p, p, i64, i64, i64, i64, p, sz, p], i32),
        "blr_forward_paths_ws": ([i64, p, p, p, p, p, p, p, i64, i64, i64, i64, p, sz, p], i32),
        "blr_backward_workspace_size": ([i64, i64, i64, i64], sz),
        "blr_backward_paths": ([i64, p, p, p, p, p, p, p, p, p, p, p, i64, i64, i64, i64, ctypes.c_float, p], i32),
        "blr_backward": ([p, p, p, p, p, p, p, p, p, p, p, i64, i64, i64, i64, ctypes.c_float, p], i32),
        "blr_backward_paths_ws": ([i64, p, p, p, p, p, p, p, p, p, p, p, i64, i64, i64, i64, ctypes.c_float, p, sz,
                                   p], i32),
        "blr_backward_ws": ([p, p, p, p, p, p, p, p, p, p, p, i64, i64, i64, i64, ctypes.c_float, p, sz, p], i32),
        "blr_saved_size": ([i64, i64, i64, i64, i64], sz),
        "blr_forward_paths_save": ([i64, p, p, p, p, p, p, p, i64, i64, i64, i64, p, sz, p], i32),
        "blr_backward_paths_saved": ([i64, p, p, p, p, p, p, p, p, p, p, p, i64, i64, i64, i64, ctypes.c_float, p, sz,
                                      p], i32),
        "tq2_strerror": ([i32], ctypes.c_char_p),
        "tq2_version": ([], ctypes.c_char_p),
    }
    sig |= {
        "q4_packed_size": ([i64, i64, i64, i64, i32], sz),
        "q4_pack": ([p, p, p, p, p], i32),
        "q4_dequant": ([p, p, p], i32),
        "q4_gemm_workspace_size": ([p, i64, i32], sz),
        "q4_gemm": ([p, p, p, i64, i32, p, sz, p], i32),
        "moe_route": ([p, p, p, p, i64, i64, i64, i64, i64, i64, i32, i32, i32, p], i32),
        "moe_route_backward": ([p, p, p, p, i64, i64, i64, i32, i32, i32, p], i32),
        "q4_moe_workspace_size": ([i64, i64, i64, i64, i64, i32], sz),
        "q4_moe": ([p, p, p, p, p, p, p, i64, i64, i32, p, sz, p], i32),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    from . import _binding as calls

    calls.bind(*(ctypes.cast(f, p).value for f in (L.q4_gemm_workspace_size, L.q4_gemm, L.moe_route, L.moe_route_backward,
                                                   L.q4_moe_workspace_size, L.q4_moe)))
    _lib, _compiled = L, calls
    return L


def _check(status: int, what: str):
    if status != TQ2_OK:
        raise Tq2Error(status, what)


def _stream(stream):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on(stream):
    """The stream as a torch stream (a raw handle is wrapped; 0 is the default stream's), or None."""
    if stream is None or hasattr(stream, "cuda_stream"):
        return stream
    import torch

    # a stream object made of the handle 0 would be a new stream of torch's pool
    return torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()


def _empty(shape, dtype, device, stream):
    """New device memory for a call on `stream` (a torch stream, or None), which the caller's current stream may
    use as well.  It comes from that stream's own pool: another's may hand out memory that work queued there still uses."""
    import torch

    if stream is None or torch.device(device).type != "cuda":  # (another device is refused where the tensor is used)
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _dev(t, dtype, name):
    import torch

    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a tensor on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def tq2_strerror(status: int) -> str:
    return lib().tq2_strerror(int(status)).decode()


def tq2_version() -> str:
    return lib().tq2_version().decode()


def tq2_select_path(m: int) -> int:
    return int(lib().tq2_select_path(int(m)))


def tq2_set_m_small(v: int) -> int:
    return int(lib().tq2_set_m_small(int(v)))


def tq2_set_path(path: int) -> int:
    """Force the path of every auto call (TQ2_PATH_AUTO restores the choice by M); returns the old setting."""
    st = int(lib().tq2_set_path(int(path)))
    if st < 0:
        raise Tq2Error(st, "tq2_set_path")
    return st


def tq2_workspace_allocs() -> int:
    """Device allocations the library has made for its own (grow-only) workspaces."""
    return int(lib().tq2_workspace_allocs())


def blr_workspace_size(m: int, d_in: int, d_out: int, r: int) -> int:
    return int(lib().blr_workspace_size(int(m), int(d_in), int(d_out), int(r)))


class Tq2Weight:
    """Device handle of an uploaded TQ2_0_g128 weight [N][K]; freed on close()/GC."""

    def __init__(self, handle: ctypes.c_void_p, n: int, k: int):
        self._h = handle
        self.N, self.K = n, k

    @property
    def handle(self):
        if self._h is None:
            raise ValueError("weight already freed")
        return self._h

    def device_bytes(self) -> int:
        nb = ctypes.c_size_t()
        _check(lib().tq2_weight_info(self.handle, None, None, ctypes.byref(nb)), "tq2_weight_info")
        return nb.value

    def close(self):
        if self._h is not None:
            h, self._h = self._h, None
            _check(lib().tq2_free(h), "tq2_free")

    def __del__(self):
        try:
            if self._h is not None and _lib is not None:
                _lib.tq2_free(self._h)
                self._h = None
        except Exception:
            pass


def tq2_upload(aos, n: int, k: int, stream=None) -> Tq2Weight:
    """Upload AoS block bytes (numpy uint8 / bytes) for a weight [n][k]."""
    buf = np.ascontiguousarray(np.frombuffer(aos, np.uint8) if isinstance(aos, (bytes, bytearray)) else aos,
                               dtype=np.uint8)
    out = ctypes.c_void_p()
    _check(lib().tq2_upload(buf.ctypes.data_as(ctypes.c_void_p), buf.size, int(n), int(k), _stream(stream),
                            ctypes.byref(out)), "tq2_upload")
    return Tq2Weight(out, int(n), int(k))


def tq2_free(w: Tq2Weight):
    w.close()


def tq2_gemm_path(w: Tq2Weight, x, y=None, path: int = TQ2_PATH_AUTO, stream=None):
    """y[M][N] = x[M][K] @ W^T on the chosen path; returns y (allocated if None)."""
    import torch

    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError(f"x must be [M, {w.K}]")
    m = x.shape[0]
    if y is None:
        y = _empty((m, w.N), torch.float32, x.device, _on(stream))
    if y.shape != (m, w.N):
        raise ValueError(f"y must be [{m}, {w.N}]")
    _check(lib().tq2_gemm_path(w.handle, _dev(x, torch.float32, "x"), _dev(y, torch.float32, "y"), m, w.N, w.K,
                               int(path), _stream(stream)), "tq2_gemm")
    return y


def tq2_gemm(w: Tq2Weight, x, y=None, stream=None):
    return tq2_gemm_path(w, x, y, TQ2_PATH_AUTO, stream)


def tq2_dequant(w: Tq2Weight, out=None, stream=None):
    import torch

    if out is None:
        out = _empty((w.N, w.K), torch.float32, "cuda", _on(stream))
    if tuple(out.shape) != (w.N, w.K):
        raise ValueError(f"out must be [{w.N}, {w.K}]")
    _check(lib().tq2_dequant(w.handle, _dev(out, torch.float32, "out"), _stream(stream)), "tq2_dequant")
    return out


def _shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _blr_sizes(bits_u, bits_v, h, l, g, x, paths: bool):
    """(P, M, d_in, d_out, r) from x, h and l, with every operand's shape checked
    against them (bits as int32 words: [P][d_out][r/32] and [P][d_in][r/32])."""
    if x.dim() != 2:
        raise ValueError("x must be [M, d_in]")
    m, d_in = x.shape
    if paths:
        if h.dim() != 2 or l.dim() != 2:
            raise ValueError("h and l must be [P, d_out] and [P, r]")
        npaths, d_out = h.shape
        r = l.shape[1]
        lead = (npaths,)
    else:
        if h.dim() != 1 or l.dim() != 1:
            raise ValueError("h and l must be [d_out] and [r]")
        npaths, d_out, r = 1, h.shape[0], l.shape[0]
        lead = ()
    if r % 32:
        raise ValueError(f"r must be a multiple of 32, got {r}")
    _shape(l, lead + (r,), "l")
    _shape(g, lead + (d_in,), "g")
    _shape(bits_u, lead + (d_out, r // 32), "bits_u")
    _shape(bits_v, lead + (d_in, r // 32), "bits_v")
    return npaths, m, d_in, d_out, r


def _workspace(workspace, need, like, stream, what):
    """A caller workspace checked for size, or a temporary one tied to `stream`."""
    import torch

    if need == 0:
        raise Tq2Error(TQ2_EINVAL, what)
    if workspace is None:
        workspace = _empty(need, torch.uint8, like.device, _on(stream))
    if workspace.numel() < need:
        raise ValueError(f"workspace needs {need} bytes, got {workspace.numel()}")
    return workspace


def _blr_forward_call(bits_u, bits_v, h, l, g, x, y, stream, paths: bool, workspace=None, use_ws=False):
    import torch

    npaths, m, d_in, d_out, r = _blr_sizes(bits_u, bits_v, h, l, g, x, paths)
    if y is None:
        y = _empty((m, d_out), torch.float32, x.device, _on(stream))
    _shape(y, (m, d_out), "y")
    args = [_dev(bits_u, torch.int32, "bits_u"), _dev(bits_v, torch.int32, "bits_v"), _dev(h, torch.float32, "h"),
            _dev(l, torch.float32, "l"), _dev(g, torch.float32, "g"), _dev(x, torch.float32, "x"),
            _dev(y, torch.float32, "y"), m, d_in, d_out, r]
    if use_ws:
        ws = _workspace(workspace, blr_workspace_size(m, d_in, d_out, r), x, stream, "blr_workspace_size")
        args += [_dev(ws, torch.uint8, "workspace"), ws.numel()]
    args.append(_stream(stream))
    L = lib()
    if paths:
        fn = L.blr_forward_paths_ws if use_ws else L.blr_forward_paths
        _check(fn(npaths, *args), fn.__name__)
    else:
        fn = L.blr_forward_ws if use_ws else L.blr_forward
        _check(fn(*args), fn.__name__)
    return y


def blr_forward(bits_u, bits_v, h, l, g, x, y=None, stream=None):
    """Binary low-rank layer forward (library-owned workspace); bits_* are int32
    tensors holding the u32 bitmap words [d_out][r/32] and [d_in][r/32]."""
    return _blr_forward_call(bits_u, bits_v, h, l, g, x, y, stream, paths=False)


def blr_forward_ws(bits_u, bits_v, h, l, g, x, y=None, workspace=None, stream=None):
    """blr_forward with a caller-owned workspace (uint8, >= blr_workspace_size bytes)."""
    return _blr_forward_call(bits_u, bits_v, h, l, g, x, y, stream, paths=False, workspace=workspace, use_ws=True)


def blr_forward_paths(bits_u, bits_v, h, l, g, x, y=None, stream=None):
    """A layer of P paths, y = sum_p h_p . c_p, rounded path by path; the per-path
    operands are stacked along a leading P axis (bits_u [P][d_out][r/32], bits_v
    [P][d_in][r/32], h [P][d_out], l [P][r], g [P][d_in])."""
    return _blr_forward_call(bits_u, bits_v, h, l, g, x, y, stream, paths=True)


def blr_forward_paths_ws(bits_u, bits_v, h, l, g, x, y=None, workspace=None, stream=None):
    return _blr_forward_call(bits_u, bits_v, h, l, g, x, y, stream, paths=True, workspace=workspace, use_ws=True)


def blr_backward_workspace_size(m: int, d_in: int, d_out: int, r: int) -> int:
    return int(lib().blr_backward_workspace_size(m, d_in, d_out, r))


def blr_saved_size(paths: int, m: int, d_in: int, d_out: int, r: int) -> int:
    return int(lib().blr_saved_size(int(paths), int(m), int(d_in), int(d_out), int(r)))


def blr_forward_paths_save(bits_u, bits_v, h, l, g, x, y=None, saved=None, stream=None):
    """blr_forward_paths that also keeps each path's a and c (f32) in `saved` (uint8,
    >= blr_saved_size bytes; allocated if None) for blr_backward_paths_saved.
    Returns (y, saved)."""
    import torch

    npaths, m, d_in, d_out, r = _blr_sizes(bits_u, bits_v, h, l, g, x, paths=True)
    if y is None:
        y = _empty((m, d_out), torch.float32, x.device, _on(stream))
    _shape(y, (m, d_out), "y")
    need = blr_saved_size(npaths, m, d_in, d_out, r)
    if need == 0:
        raise Tq2Error(TQ2_EINVAL, "blr_saved_size")
    if saved is None:
        saved = _empty(need, torch.uint8, x.device, _on(stream))
    if saved.dim() != 1 or saved.numel() < need:
        raise ValueError(f"saved must be a flat uint8 tensor of at least {need} bytes")
    _check(lib().blr_forward_paths_save(
        npaths, _dev(bits_u, torch.int32, "bits_u"), _dev(bits_v, torch.int32, "bits_v"),
        _dev(h, torch.float32, "h"), _dev(l, torch.float32, "l"), _dev(g, torch.float32, "g"),
        _dev(x, torch.float32, "x"), _dev(y, torch.float32, "y"), m, d_in, d_out, r,
        _dev(saved, torch.uint8, "saved"), saved.numel(), _stream(stream)), "blr_forward_paths_save")
    return y, saved


def blr_saved_views(saved, paths: int, m: int, d_out: int, r: int):
    """Per-path views (a [M][r], c [M][d_out]) of a buffer filled by blr_forward_paths_save."""
    import torch

    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    a_bytes = up(m * r * 4)
    path_bytes = a_bytes + up(m * d_out * 4)
    out = []
    for q in range(paths):
        base = q * path_bytes
        a = saved[base: base + m * r * 4].view(torch.float32).view(m, r)
        c = saved[base + a_bytes: base + a_bytes + m * d_out * 4].view(torch.float32).view(m, d_out)
        out.append((a, c))
    return out


def blr_backward_paths_saved(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, saved, dx=None, gscale=1024.0,
                             stream=None):
    """blr_backward_paths from the activations blr_forward_paths_save kept in `saved`
    (same layer and x): no recomputation, the same bits."""
    return _blr_backward_call(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, dx, gscale, stream, None, False,
                              saved=saved)


def _blr_backward_call(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, dx, gscale, stream, workspace, use_ws,
                       saved=None):
    import torch

    npaths, m, d_in, d_out, r = _blr_sizes(bits_u, bits_v, h, l, g, x, paths=True)
    _shape(dy, (m, d_out), "dy")
    _shape(dh, (npaths, d_out), "dh")
    _shape(dl, (npaths, r), "dl")
    _shape(dg, (npaths, d_in), "dg")
    if dx is None:
        dx = _empty((m, d_in), torch.float32, x.device, _on(stream))
    _shape(dx, (m, d_in), "dx")
    args = [npaths, _dev(bits_u, torch.int32, "bits_u"), _dev(bits_v, torch.int32, "bits_v"),
            _dev(h, torch.float32, "h"), _dev(l, torch.float32, "l"), _dev(g, torch.float32, "g"),
            _dev(x, torch.float32, "x"), _dev(dy, torch.float32, "dy"), _dev(dx, torch.float32, "dx"),
            _dev(dh, torch.float32, "dh"), _dev(dl, torch.float32, "dl"), _dev(dg, torch.float32, "dg"),
            m, d_in, d_out, r, float(gscale)]
    L = lib()
    if saved is not None:
        need = blr_saved_size(npaths, m, d_in, d_out, r)
        if saved.dim() != 1 or saved.numel() < need:
            raise ValueError(f"saved must be a flat uint8 tensor of at least {need} bytes")
        _check(L.blr_backward_paths_saved(*args, _dev(saved, torch.uint8, "saved"), saved.numel(),
                                          _stream(stream)), "blr_backward_paths_saved")
    elif use_ws:
        ws = _workspace(workspace, blr_backward_workspace_size(m, d_in, d_out, r), x, stream,
                        "blr_backward_workspace_size")
        _check(L.blr_backward_paths_ws(*args, _dev(ws, torch.uint8, "workspace"), ws.numel(), _stream(stream)),
               "blr_backward_paths_ws")
    else:
        _check(L.blr_backward_paths(*args, _stream(stream)), "blr_backward_paths")
    return dx


def blr_backward_paths(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, dx=None, gscale=1024.0, stream=None):
    """Backward of blr_forward_paths on the same x (library-owned workspace): dh [P][d_out],
    dl [P][r] and dg [P][d_in] are accumulated in place; dx [M][d_in] is overwritten (returned)."""
    return _blr_backward_call(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, dx, gscale, stream, None, False)


def blr_backward_paths_ws(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, dx=None, gscale=1024.0, workspace=None,
                          stream=None):
    """blr_backward_paths with a caller-owned workspace (uint8, >= blr_backward_workspace_size bytes)."""
    return _blr_backward_call(bits_u, bits_v, h, l, g, x, dy, dh, dl, dg, dx, gscale, stream, workspace, True)


# ---------------------------------------------------------------- 4-bit weights and mixtures of experts

Q4_F32, Q4_F16, Q4_BF16 = 0, 1, 2
MOE_SOFTMAX, MOE_SIGMOID = 0, 1
_SCORES = {"softmax": MOE_SOFTMAX, "sigmoid": MOE_SIGMOID}
_compiled = None  # the calls' tensor checks and marshalling (csrc/binding.cpp); set by lib()


def _calls():
    """The compiled calls, bound to the library's entry points."""
    lib()
    return _compiled


def _for(stream, *tensors):
    """The stream as a torch stream, or None; tensors that a call on it takes keep their memory until it is done with them."""
    if stream is None:
        return None
    import torch

    s = _on(stream)
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(s)
    return s


class _Q4Struct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("E", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("G", ctypes.c_int64), ("zeros", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class Q4Weight:
    """A packed 4-bit weight [N][K] (E is None) or stack of them [E][N][K]; its memory is a torch tensor."""

    def __init__(self, data, e, n, k, g, zeros: bool):
        self.data, self.E, self.N, self.K, self.G, self.zeros = data, e, n, k, g, zeros
        self.like = (e, n, k, g, zeros)
        self.device = data.get_device()
        self._struct = _Q4Struct(data.data_ptr(), 1 if e is None else e, n, k, g, int(zeros), 0)
        self.handle = ctypes.addressof(self._struct)

    def device_bytes(self) -> int:
        return self.data.numel()


def q4_upload(codes, scales, zeros=None, stream=None) -> Q4Weight:
    """Pack a 4-bit weight: codes uint8 [..., N, K/2] (element 2j in the low four bits of byte j), scales float16
    [..., N, K/G] with G 32, 64 or 128, zeros uint8 like scales (8 everywhere if None); W = (code - zero) * scale.
    `...` is nothing, or one axis of experts.  As in all calls below, `stream` is a torch stream or a raw handle (None: the
    current stream); tensors given to a call may be freed at once, their memory stays until the stream is done with it."""
    import torch

    if codes.dim() not in (2, 3) or codes.numel() == 0:
        raise ValueError("codes must be [N, K/2] or [E, N, K/2], and not empty")
    e = codes.shape[0] if codes.dim() == 3 else None
    n, k = codes.shape[-2], 2 * codes.shape[-1]
    if scales.dim() != codes.dim() or scales.shape[-1] == 0 or k % scales.shape[-1]:
        raise ValueError(f"scales must be [{'E, ' if e is not None else ''}{n}, K/G], got {tuple(scales.shape)}")
    g = k // scales.shape[-1]
    need = lib().q4_packed_size(e or 1, n, k, g, int(zeros is not None))
    if need == 0:
        raise ValueError(f"no packed form for E={e}, N={n}, K={k}, G={g}: G is 32, 64 or 128 and divides K")
    c, lead, stream = _calls(), codes.shape[:-1], _for(stream, codes, scales, zeros)
    pc = c.address(codes, "u8", codes.shape, "codes", None)
    device = codes.get_device()
    ps = c.address(scales, "f16", (*lead, k // g), "scales", device)
    pz = None if zeros is None else c.address(zeros, "u8", (*lead, k // g), "zeros", device)
    raw = c.stream(stream, device)
    w = Q4Weight(_empty(need, torch.uint8, codes.device, stream), e, n, k, g, zeros is not None)
    _check(lib().q4_pack(w.handle, pc, ps, pz, raw), "q4_pack")
    return w


def q4_dequant(w: Q4Weight, out=None, stream=None):
    """(code - zero) * scale as float32, exact: [N, K] or [E, N, K]."""
    import torch

    c, stream = _calls(), _for(stream, w.data, out)
    shape = (w.N, w.K) if w.E is None else (w.E, w.N, w.K)
    raw = c.stream(stream, w.device)
    if out is None:
        out = _empty(shape, torch.float32, w.data.device, stream)
    _check(lib().q4_dequant(w.handle, c.address(out, "f32", shape, "out", w.device), raw), "q4_dequant")
    return out


def q4_gemm(w: Q4Weight, x, y=None, stream=None):
    """y[M][N] = x[M][K] @ W^T in x's type (float32, float16 or bfloat16); returns y (allocated if None)."""
    if w.E is not None:
        raise ValueError("q4_gemm takes a weight without an axis of experts")
    out = (_compiled or _calls()).gemm(w.handle, w.device, x, y, stream if stream is None else _for(stream, w.data, x, y))
    if out.__class__ is int:
        _check(out, "q4_gemm")
    return out


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return _SCORES[score]


def moe_route(logits, k, bias=None, score="softmax", groups=1, keep=1, group_top=1, renorm=False, idx=None,
              weights=None, stream=None):
    """Router of a mixture of experts: (idx int32 [T][k], weights float32 [T][k]) from logits [T][E] (float32,
    float16 or bfloat16).  Experts are ranked by score + bias (bias float32 [E]), within the `keep` of `groups`
    equal groups whose `group_top` best keys add up to most; equal keys go to the lower index.  The weights are the scores,
    divided by their sum if renorm.  Slots that find no expert (logits of -inf) get idx -1 and weight 0."""
    out = (_compiled or _calls()).route(logits, k, bias, _score(score), groups, keep, group_top, renorm, idx, weights,
                                       stream if stream is None else _for(stream, logits, bias, idx, weights))
    if out.__class__ is int:
        _check(out, "moe_route")
    return out


def moe_route_backward(logits, idx, dw, score="softmax", renorm=False, dlogits=None, stream=None):
    """Gradient of moe_route's weights: dlogits [T][E] (logits' type, overwritten; allocated if None) from dw
    float32 [T][k] and the idx that moe_route gave, the choice held fixed."""
    out = (_compiled or _calls()).route_backward(logits, idx, dw, _score(score), renorm, dlogits,
                                                stream if stream is None else _for(stream, logits, idx, dw, dlogits))
    if out.__class__ is int:
        _check(out, "moe_route_backward")
    return out


def q4_moe(x, idx, weights, gate: Q4Weight, up: Q4Weight, down: Q4Weight, y=None, stream=None):
    """Experts' gated products, y[t] = sum_j weights[t][j] * down_e(silu(gate_e x_t) * (up_e x_t)) with e = idx[t][j]:
    x [T][d] (float32, float16 or bfloat16), idx int32 [T][k] (entries outside 0 .. E-1 are dropped), weights float32
    [T][k], gate and up [E][f][d], down [E][d][f]; returns y [T][d] in x's type (allocated if None)."""
    if gate.E is None or up.E is None or down.E is None:
        raise ValueError("q4_moe takes weights with an axis of experts")
    if up.like != gate.like or (down.E, down.N, down.K) != (gate.E, gate.K, gate.N):
        raise ValueError(f"gate and up must be alike and down [{gate.E}, {gate.K}, {gate.N}]")
    if up.device != gate.device or down.device != gate.device:
        raise ValueError("the weights are on different devices")
    out = (_compiled or _calls()).moe(x, idx, weights, gate.handle, up.handle, down.handle, gate.device, y,
                                     stream if stream is None else
                                     _for(stream, x, idx, weights, gate.data, up.data, down.data, y))
    if out.__class__ is int:
        _check(out, "q4_moe")
    return out
