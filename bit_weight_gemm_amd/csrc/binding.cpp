// Python calls of the 4-bit weights, the mixture-of-experts operators and a block's norms.
//
// A small kernel takes a few microseconds, as long as a call whose dozen arguments are
// checked and converted in Python (6.0-7.1 us of host time for one launch; from here 3.0-3.9).
// This module checks the tensors of a call, allocates what the caller left out and calls
// the C entry points, whose addresses `bind` gets from the binding.  Host code only.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>

#include "../../include/libtq2_block.h"

namespace {

decltype(&q4_gemm_workspace_size) p_gemm_ws;
decltype(&q4_gemm) p_gemm;
decltype(&moe_route) p_route;
decltype(&moe_route_backward) p_route_backward;
decltype(&q4_moe_workspace_size) p_moe_ws;
decltype(&q4_moe) p_moe;
decltype(&q4_linear) p_linear;
decltype(&moe_layer_workspace_size) p_layer_ws;
decltype(&moe_layer) p_layer;
decltype(&block_norm) p_block;
decltype(&block_norm_backward_workspace_size) p_block_backward_ws;
decltype(&block_norm_backward) p_block_backward;

struct Refused {};  // a Python error is set

template <typename... A>
[[noreturn]] void refuse(PyObject *type, const char *format, A... a) {
    PyErr_Format(type, format, a...);
    throw Refused{};
}

const char *name_of(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kByte: return "torch.uint8";
        case at::kInt: return "torch.int32";
        default: return c10::toString(t);
    }
}

std::string text(at::IntArrayRef s) {
    std::string out = "(";
    for (size_t i = 0; i < s.size(); ++i) out += (i ? ", " : "") + std::to_string(s[i]);
    return out + ")";
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor on the GPU", name);
    return THPVariable_Unpack(o);
}

int type_code(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat) return Q4_F32;
    if (t.scalar_type() == at::kHalf) return Q4_F16;
    if (t.scalar_type() == at::kBFloat16) return Q4_BF16;
    refuse(PyExc_TypeError, "%s must be float32, float16 or bfloat16, got %s", name, name_of(t.scalar_type()));
}

int gpu_of(const at::Tensor &t, const char *name) {
    if (!t.is_cuda()) refuse(PyExc_TypeError, "%s must be a tensor on the GPU", name);
    return t.get_device();
}

// Address of a contiguous tensor of this type and shape on GPU `device`.
void *address(const at::Tensor &t, at::ScalarType type, at::IntArrayRef shape, const char *name, int device) {
    const int on = gpu_of(t, name);
    if (t.scalar_type() != type)
        refuse(PyExc_TypeError, "%s must be %s, got %s", name, name_of(type), name_of(t.scalar_type()));
    if (t.sizes() != shape)
        refuse(PyExc_ValueError, "%s must have shape %s, got %s", name, text(shape).c_str(), text(t.sizes()).c_str());
    if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
    if (on != device) refuse(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d", name, on, device);
    return t.data_ptr();
}

// The handle of a torch stream; None: the current stream of `device`, which has to be the current device.
void *raw_stream(PyObject *stream, int device) {
    const int current = c10::hip::current_device();
    if (device != current)
        refuse(PyExc_ValueError, "the tensors are on cuda:%d, the current device is cuda:%d", device, current);
    if (stream == Py_None) return c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    PyObject *handle = PyObject_GetAttrString(stream, "cuda_stream");
    if (!handle) throw Refused{};
    void *p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (PyErr_Occurred()) throw Refused{};
    return p;
}

// The calls record nothing for autograd.  Where it would want a gradient, they say so.
void no_gradient(const at::Tensor &t, const char *what) {
    if (!t.requires_grad() || !at::GradMode::is_enabled()) return;
    if (PyErr_WarnEx(PyExc_UserWarning, what, 2)) throw Refused{};
}

// New device memory for a call on `stream`.  It comes from that stream's own pool: another
// stream's may hand out memory that work queued there still uses.
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like, void *stream) {
    const at::TensorOptions options = like.options().dtype(type).requires_grad(false);
    const auto device = (c10::DeviceIndex)like.get_device();
    const c10::hip::HIPStream current = c10::hip::getCurrentHIPStream(device);
    if (current.stream() == stream) return at::empty(shape, options);
    struct Restore {
        const c10::hip::HIPStream &to;
        ~Restore() { c10::hip::setCurrentHIPStream(to); }
    } restore{current};
    c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal(static_cast<hipStream_t>(stream), device));
    return at::empty(shape, options);
}

// The tensor o, or if that is None a new one.  A new one is given to the caller's current stream
// as well, whose work on it has to end before its memory is used again.
at::Tensor output(PyObject *o, at::IntArrayRef shape, at::ScalarType type, const at::Tensor &like, const char *name,
                  void *stream) {
    if (o != Py_None) return tensor(o, name);
    at::Tensor t = fresh(shape, type, like, stream);
    const c10::hip::HIPStream current = c10::hip::getCurrentHIPStream((c10::DeviceIndex)like.get_device());
    if (current.stream() != stream) t.record_stream(c10::Stream(c10::Stream::UNSAFE, t.device(), current.id()));
    return t;
}

// A temporary workspace.
at::Tensor scratch(size_t need, const at::Tensor &like, void *stream) {
    return fresh({(int64_t)need}, at::kByte, like, stream);
}

int64_t number(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

const q4_weight *weight(PyObject *handle) {
    void *p = PyLong_AsVoidPtr(handle);
    if (PyErr_Occurred()) throw Refused{};
    if (!p) refuse(PyExc_ValueError, "no weight%s", "");
    return static_cast<const q4_weight *>(p);
}

// The entry point's status as a number, or the output tensors.
template <typename F>
int call(F &&f) {
    PyThreadState *state = PyEval_SaveThread();
    const int st = f();
    PyEval_RestoreThread(state);
    return st;
}

PyObject *result(int st, const at::Tensor &t) { return st ? PyLong_FromLong(st) : THPVariable_Wrap(t); }

void count(Py_ssize_t n, Py_ssize_t want) {
    if (n != want) refuse(PyExc_TypeError, "%zd arguments, not %zd", n, want);
}

// Runs body(args); C++ exceptions become Python ones.
template <typename F>
PyObject *guarded(F &&body) {
    HANDLE_TH_ERRORS
    try {
        return body();
    } catch (const Refused &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 12);
        auto at = [&](int i) { return PyLong_AsVoidPtr(a[i]); };
        p_gemm_ws = reinterpret_cast<decltype(p_gemm_ws)>(at(0));
        p_gemm = reinterpret_cast<decltype(p_gemm)>(at(1));
        p_route = reinterpret_cast<decltype(p_route)>(at(2));
        p_route_backward = reinterpret_cast<decltype(p_route_backward)>(at(3));
        p_moe_ws = reinterpret_cast<decltype(p_moe_ws)>(at(4));
        p_moe = reinterpret_cast<decltype(p_moe)>(at(5));
        p_linear = reinterpret_cast<decltype(p_linear)>(at(6));
        p_layer_ws = reinterpret_cast<decltype(p_layer_ws)>(at(7));
        p_layer = reinterpret_cast<decltype(p_layer)>(at(8));
        p_block = reinterpret_cast<decltype(p_block)>(at(9));
        p_block_backward_ws = reinterpret_cast<decltype(p_block_backward_ws)>(at(10));
        p_block_backward = reinterpret_cast<decltype(p_block_backward)>(at(11));
        if (PyErr_Occurred()) throw Refused{};
        Py_RETURN_NONE;
    });
}

// address(tensor, type, shape, name, device), type: "u8", "f16" or "f32"
PyObject *py_address(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 5);
        const char *name = PyUnicode_AsUTF8(a[3]), *type = PyUnicode_AsUTF8(a[1]);
        if (!name || !type) throw Refused{};
        const at::ScalarType t = type[0] == 'u' ? at::kByte : type[1] == '1' ? at::kHalf : at::kFloat;
        std::vector<int64_t> shape;
        PyObject *s = PySequence_Fast(a[2], "a shape");
        if (!s) throw Refused{};
        for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(s); ++i)
            shape.push_back(PyLong_AsLongLong(PySequence_Fast_GET_ITEM(s, i)));
        Py_DECREF(s);
        if (PyErr_Occurred()) throw Refused{};
        const int device = a[4] == Py_None ? gpu_of(tensor(a[0], name), name) : (int)number(a[4]);
        return PyLong_FromVoidPtr(address(tensor(a[0], name), t, shape, name, device));
    });
}

// stream(stream or None, device): its handle
PyObject *py_stream(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 2);
        return PyLong_FromVoidPtr(raw_stream(a[0], (int)number(a[1])));
    });
}

// gemm(handle, device, x, y, stream)
PyObject *py_gemm(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 5);
        const q4_weight *w = weight(a[0]);
        const int device = (int)number(a[1]);
        const at::Tensor &x = tensor(a[2], "x");
        if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [M, %lld]", (long long)w->K);
        const int64_t m = x.size(0);
        const int code = type_code(x, "x");
        const void *px = address(x, x.scalar_type(), {m, w->K}, "x", device);
        no_gradient(x, "q4_gemm forms no gradient, but x requires one (detach it, or call under torch.no_grad())");
        void *stream = raw_stream(a[4], device);
        const at::Tensor y = output(a[3], {m, w->N}, x.scalar_type(), x, "y", stream);
        void *py = address(y, x.scalar_type(), {m, w->N}, "y", device);
        const size_t need = p_gemm_ws(w, m, code);
        at::Tensor ws;
        if (need) ws = scratch(need, x, stream);
        void *pw = need ? ws.data_ptr() : nullptr;
        return result(call([&] { return p_gemm(w, px, py, m, code, pw, need, stream); }), y);
    });
}

// route(logits, k, bias, score, groups, keep, group_top, renorm, idx, weights, stream)
PyObject *py_route(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 11);
        const at::Tensor &l = tensor(a[0], "logits");
        if (l.dim() != 2) refuse(PyExc_ValueError, "logits must be [T, E]%s", "");
        const int64_t t = l.size(0), e = l.size(1), k = number(a[1]);
        const int code = type_code(l, "logits"), score = (int)number(a[3]), renorm = truth(a[7]);
        const int64_t groups = number(a[4]), keep = number(a[5]), group_top = number(a[6]);
        if (k < 1 || k > e || k > 64)
            refuse(PyExc_ValueError, "k must lie between 1 and %lld, got %lld", (long long)(e < 64 ? e : 64), (long long)k);
        if (e > 1024 || groups < 1 || groups > 64 || e % groups || keep < 1 || keep > groups || group_top < 1 || group_top > 2)
            refuse(PyExc_ValueError, "no routing over E=%lld, groups=%lld, keep=%lld, group_top=%lld", (long long)e,
                   (long long)groups, (long long)keep, (long long)group_top);
        const int device = gpu_of(l, "logits");
        const void *pl = address(l, l.scalar_type(), {t, e}, "logits", device);
        no_gradient(l, "moe_route records no gradient, but logits require one: it comes from moe_route_backward (call moe_route "
                       "under torch.no_grad())");
        const void *pb = a[2] == Py_None ? nullptr : address(tensor(a[2], "bias"), at::kFloat, {e}, "bias", device);
        void *stream = raw_stream(a[10], device);
        const at::Tensor idx = output(a[8], {t, k}, at::kInt, l, "idx", stream);
        const at::Tensor w = output(a[9], {t, k}, at::kFloat, l, "weights", stream);
        void *pi = address(idx, at::kInt, {t, k}, "idx", device), *pw = address(w, at::kFloat, {t, k}, "weights", device);
        const int st = call([&] {
            return p_route(pl, static_cast<const float *>(pb), static_cast<int32_t *>(pi), static_cast<float *>(pw), t, e, k,
                           groups, keep, group_top, score, renorm, code, stream);
        });
        if (st) return PyLong_FromLong(st);
        return Py_BuildValue("NN", THPVariable_Wrap(idx), THPVariable_Wrap(w));
    });
}

// route_backward(logits, idx, dw, score, renorm, dlogits, stream)
PyObject *py_route_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 7);
        const at::Tensor &l = tensor(a[0], "logits"), &idx = tensor(a[1], "idx"), &dw = tensor(a[2], "dw");
        if (l.dim() != 2 || idx.dim() != 2) refuse(PyExc_ValueError, "logits must be [T, E] and idx [T, k]%s", "");
        const int64_t t = l.size(0), e = l.size(1), k = idx.size(1);
        const int code = type_code(l, "logits"), score = (int)number(a[3]), renorm = truth(a[4]);
        if (k < 1 || k > 64 || e < 1 || e > 1024)
            refuse(PyExc_ValueError, "no routing of k=%lld out of E=%lld", (long long)k, (long long)e);
        const int device = gpu_of(l, "logits");
        const void *pl = address(l, l.scalar_type(), {t, e}, "logits", device);
        const void *pi = address(idx, at::kInt, {t, k}, "idx", device), *pw = address(dw, at::kFloat, {t, k}, "dw", device);
        void *stream = raw_stream(a[6], device);
        const at::Tensor dl = output(a[5], {t, e}, l.scalar_type(), l, "dlogits", stream);
        void *pd = address(dl, l.scalar_type(), {t, e}, "dlogits", device);
        return result(call([&] {
                          return p_route_backward(pl, static_cast<const int32_t *>(pi), static_cast<const float *>(pw), pd, t,
                                                  e, k, score, renorm, code, stream);
                      }),
                      dl);
    });
}

// moe(x, idx, weights, gate, up, down, device, y, stream): handles of the three weights
PyObject *py_moe(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 9);
        const at::Tensor &x = tensor(a[0], "x"), &idx = tensor(a[1], "idx"), &wts = tensor(a[2], "weights");
        const q4_weight *gate = weight(a[3]), *up = weight(a[4]), *down = weight(a[5]);
        if (x.dim() != 2 || idx.dim() != 2) refuse(PyExc_ValueError, "x must be [T, d] and idx [T, k]%s", "");
        const int64_t t = idx.size(0), k = idx.size(1), e = gate->E, f = gate->N, d = gate->K;
        const int code = type_code(x, "x"), device = (int)number(a[6]);
        const void *px = address(x, x.scalar_type(), {t, d}, "x", device);
        const void *pi = address(idx, at::kInt, {t, k}, "idx", device);
        const void *pw = address(wts, at::kFloat, {t, k}, "weights", device);
        no_gradient(x, "q4_moe forms no gradients, but x requires one (detach it, or call under torch.no_grad())");
        no_gradient(wts, "q4_moe forms no gradients, but weights require one (detach them, or call under torch.no_grad())");
        void *stream = raw_stream(a[8], device);
        const at::Tensor y = output(a[7], {t, d}, x.scalar_type(), x, "y", stream);
        void *py = address(y, x.scalar_type(), {t, d}, "y", device);
        const size_t need = p_moe_ws(t, k, e, d, f, code);
        if (need == 0)
            refuse(PyExc_ValueError, "no experts' products for T=%lld, k=%lld, E=%lld, d=%lld, f=%lld", (long long)t,
                   (long long)k, (long long)e, (long long)d, (long long)f);
        const at::Tensor ws = scratch(need, x, stream);
        void *pws = ws.data_ptr();
        return result(call([&] {
                          return p_moe(px, static_cast<const int32_t *>(pi), static_cast<const float *>(pw), gate, up, down, py,
                                       t, k, code, pws, need, stream);
                      }),
                      y);
    });
}

double real(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return v;
}

// Address of a tensor that a call may go without (None: nullptr).
void *maybe(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name, int device) {
    return o == Py_None ? nullptr : address(tensor(o, name), type, shape, name, device);
}

// A parameter vector, of float32 or the rows' type; `code` is set to its type.
void *side(PyObject *o, const at::Tensor &rows, at::IntArrayRef shape, const char *name, int device, int &code) {
    if (o == Py_None) return nullptr;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != rows.scalar_type())
        refuse(PyExc_TypeError, "%s must be torch.float32 or %s, got %s", name, name_of(rows.scalar_type()), name_of(t.scalar_type()));
    code = type_code(t, name);
    return address(t, t.scalar_type(), shape, name, device);
}

void no_gradient(PyObject *o, const char *name, const char *what) {
    if (o != Py_None) no_gradient(tensor(o, name), what);
}

// linear(handle, device, x, bias, activation, residual, y, stream)
PyObject *py_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 8);
        const q4_weight *w = weight(a[0]);
        const int device = (int)number(a[1]), act = (int)number(a[4]);
        const at::Tensor &x = tensor(a[2], "x");
        if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [M, %lld]", (long long)w->K);
        const int64_t m = x.size(0);
        const int code = type_code(x, "x");
        int bias_code = code;
        const void *px = address(x, x.scalar_type(), {m, w->K}, "x", device);
        const void *pb = side(a[3], x, {w->N}, "bias", device, bias_code);
        const void *pr = maybe(a[5], x.scalar_type(), {m, w->N}, "residual", device);
        constexpr const char *kNo = "q4_linear forms no gradient, but an argument requires one (detach it, or call under torch.no_grad())";
        no_gradient(x, kNo), no_gradient(a[3], "bias", kNo), no_gradient(a[5], "residual", kNo);
        void *stream = raw_stream(a[7], device);
        const at::Tensor y = output(a[6], {m, w->N}, x.scalar_type(), x, "y", stream);
        void *py = address(y, x.scalar_type(), {m, w->N}, "y", device);
        const size_t need = p_gemm_ws(w, m, code);
        at::Tensor ws;
        if (need) ws = scratch(need, x, stream);
        void *pw = need ? ws.data_ptr() : nullptr;
        return result(call([&] { return p_linear(w, px, pb, bias_code, act, pr, py, m, code, pw, need, stream); }), y);
    });
}

// layer(x, router, gate, up, down, device, k, norm, eps, bias, score, groups, keep, group_top, renorm, residual, y, idx, weights,
//       stream): handles of the three weights
PyObject *py_layer(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 20);
        const at::Tensor &x = tensor(a[0], "x");
        moe_layer_call c{};
        c.gate = weight(a[2]), c.up = weight(a[3]), c.down = weight(a[4]);
        const int device = (int)number(a[5]);
        const int64_t e = c.gate->E, f = c.gate->N, d = c.gate->K;
        if (x.dim() != 2) refuse(PyExc_ValueError, "x must be [T, %lld]", (long long)d);
        const int64_t t = x.size(0);
        c.T = t, c.k = number(a[6]), c.groups = number(a[11]), c.keep = number(a[12]), c.group_top = number(a[13]);
        c.score = (int)number(a[10]), c.renorm = truth(a[14]), c.dtype = type_code(x, "x"), c.eps = real(a[8]);
        if (c.k < 1 || c.k > e || c.k > 64)
            refuse(PyExc_ValueError, "k must lie between 1 and %lld, got %lld", (long long)(e < 64 ? e : 64), (long long)c.k);
        if (c.groups < 1 || c.groups > 64 || e % c.groups || c.keep < 1 || c.keep > c.groups || c.group_top < 1 || c.group_top > 2)
            refuse(PyExc_ValueError, "no routing over E=%lld, groups=%lld, keep=%lld, group_top=%lld", (long long)e,
                   (long long)c.groups, (long long)c.keep, (long long)c.group_top);
        const at::ScalarType type = x.scalar_type();
        c.x = address(x, type, {t, d}, "x", device);
        if (a[1] == Py_None) refuse(PyExc_TypeError, "router must be a tensor on the GPU%s", "");
        c.router = side(a[1], x, {e, d}, "router", device, c.router_dtype);
        c.norm = side(a[7], x, {d}, "norm", device, c.norm_dtype);
        c.bias = static_cast<const float *>(maybe(a[9], at::kFloat, {e}, "bias", device));
        c.residual = maybe(a[15], type, {t, d}, "residual", device);
        constexpr const char *kNo = "moe_layer forms no gradients, but an argument requires one (detach it, or call under torch.no_grad())";
        no_gradient(x, kNo), no_gradient(a[1], "router", kNo), no_gradient(a[7], "norm", kNo);
        no_gradient(a[9], "bias", kNo), no_gradient(a[15], "residual", kNo);
        void *stream = raw_stream(a[19], device);
        const at::Tensor y = output(a[16], {t, d}, type, x, "y", stream);
        const at::Tensor idx = output(a[17], {t, c.k}, at::kInt, x, "idx", stream);
        const at::Tensor wts = output(a[18], {t, c.k}, at::kFloat, x, "weights", stream);
        c.y = address(y, type, {t, d}, "y", device);
        c.idx = static_cast<int32_t *>(address(idx, at::kInt, {t, c.k}, "idx", device));
        c.weights = static_cast<float *>(address(wts, at::kFloat, {t, c.k}, "weights", device));
        const size_t need = p_layer_ws(t, c.k, e, d, f, c.dtype, c.norm != nullptr);
        if (need == 0)
            refuse(PyExc_ValueError, "no layer for T=%lld, k=%lld, E=%lld, d=%lld, f=%lld", (long long)t, (long long)c.k,
                   (long long)e, (long long)d, (long long)f);
        const at::Tensor ws = scratch(need, x, stream);
        void *pws = ws.data_ptr();
        const int st = call([&] { return p_layer(&c, pws, need, stream); });
        if (st) return PyLong_FromLong(st);
        return Py_BuildValue("NNN", THPVariable_Wrap(y), THPVariable_Wrap(idx), THPVariable_Wrap(wts));
    });
}

// The norms' parameters, all of one type: [N], the gate [R, N].
struct Parameters {
    const void *at[5];  // post, post_bias, gate, pre, pre_bias
    int64_t rows = 1;   // R
    int code = -1;
    Parameters(PyObject *const *a, const at::Tensor &x, int device) {
        constexpr const char *names[5] = {"post", "post_bias", "gate", "pre", "pre_bias"};
        const int64_t m = x.size(0), n = x.size(1);
        for (int i = 0; i < 5; ++i) {
            at[i] = nullptr;
            if (a[i] == Py_None) continue;
            const at::Tensor &t = tensor(a[i], names[i]);
            int mine = 0;
            if (i == 2) {
                if (t.dim() != 2 || t.size(0) < 1 || (m % t.size(0)))
                    refuse(PyExc_ValueError, "gate must be [R, %lld], where R divides %lld rows", (long long)n, (long long)m);
                rows = t.size(0);
                at[i] = side(a[i], x, {rows, n}, names[i], device, mine);
            } else {
                at[i] = side(a[i], x, {n}, names[i], device, mine);
            }
            if (code >= 0 && mine != code)
                refuse(PyExc_TypeError, "%s must have the type of the other norms' weights and the gate", names[i]);
            code = mine;
        }
        if (code < 0) code = type_code(x, "x");
    }
};

// Rows without gradient; x [M, N] on a GPU.
int64_t norm_rows(const at::Tensor &x, const char *name) {
    if (x.dim() != 2) refuse(PyExc_ValueError, "%s must be [M, N]", name);
    if (x.size(1) < 1 || x.size(1) > 16384)
        refuse(PyExc_ValueError, "rows must have 1 to 16384 columns, got %lld", (long long)x.size(1));
    return x.size(0);
}

// block(x, b, post, post_bias, gate, pre, pre_bias, scale, layer, eps, y, n, stream)
PyObject *py_block(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 13);
        const at::Tensor &x = tensor(a[0], "x");
        block_norm_call c{};
        const int64_t m = norm_rows(x, "x"), cols = x.size(1);
        const int device = gpu_of(x, "x");
        const at::ScalarType type = x.scalar_type();
        c.dtype = type_code(x, "x");
        c.x = address(x, type, {m, cols}, "x", device);
        c.b = maybe(a[1], type, {m, cols}, "b", device);
        const Parameters p(a + 2, x, device);
        c.post = p.at[0], c.post_bias = p.at[1], c.gate = p.at[2], c.pre = p.at[3], c.pre_bias = p.at[4];
        c.M = m, c.N = cols, c.R = p.rows, c.weights_dtype = p.code;
        c.scale = (float)real(a[7]), c.layer = truth(a[8]), c.eps = real(a[9]);
        const bool b = a[1] != Py_None, pre = a[5] != Py_None;  // (tensors without rows have no address)
        if (!b && (c.post || c.gate || a[10] != Py_None)) refuse(PyExc_ValueError, "post, gate and y go with b%s", "");
        if ((!c.post && c.post_bias) || (!pre && (c.pre_bias || a[11] != Py_None)))
            refuse(PyExc_ValueError, "post_bias goes with post, pre_bias and n with pre%s", "");
        if (!b && !pre) refuse(PyExc_ValueError, "there is neither b nor pre: nothing to do%s", "");
        constexpr const char *kNo = "block_norm records no gradient, but an argument requires one: it comes from block_norm_backward "
                                    "(call block_norm under torch.no_grad())";
        constexpr const char *names[7] = {"x", "b", "post", "post_bias", "gate", "pre", "pre_bias"};
        for (int i = 0; i < 7; ++i) no_gradient(a[i], names[i], kNo);
        void *stream = raw_stream(a[12], device);
        at::Tensor y, out;
        if (b) {
            y = output(a[10], {m, cols}, type, x, "y", stream);
            c.y = address(y, type, {m, cols}, "y", device);
        }
        if (pre) {
            out = output(a[11], {m, cols}, type, x, "n", stream);
            c.n = address(out, type, {m, cols}, "n", device);
        }
        const int st = call([&] { return p_block(&c, stream); });
        if (st) return PyLong_FromLong(st);
        PyObject *first = THPVariable_Wrap(b ? y : x);
        if (pre) return Py_BuildValue("NN", first, THPVariable_Wrap(out));
        return Py_BuildValue("NO", first, Py_None);
    });
}

// block_backward(dy, y, dn, b, post, post_bias, gate, pre, pre_bias, scale, layer, eps, dx, db, stream): a dict
PyObject *py_block_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded([&]() -> PyObject * {
        count(n, 15);
        if (a[0] == Py_None && a[2] == Py_None) refuse(PyExc_ValueError, "there is neither dy nor dn%s", "");
        const at::Tensor &x = a[0] == Py_None ? tensor(a[2], "dn") : tensor(a[0], "dy");
        block_norm_backward_call c{};
        const int64_t m = norm_rows(x, "dy"), cols = x.size(1);
        const int device = gpu_of(x, "dy");
        const at::ScalarType type = x.scalar_type();
        c.dtype = type_code(x, "dy");
        const std::array<int64_t, 2> rows{m, cols};
        c.dy = maybe(a[0], type, rows, "dy", device), c.dn = maybe(a[2], type, rows, "dn", device);
        c.b = maybe(a[3], type, rows, "b", device);
        const Parameters p(a + 4, x, device);
        c.post = p.at[0], c.post_bias = p.at[1], c.gate = p.at[2], c.pre = p.at[3], c.pre_bias = p.at[4];
        c.M = m, c.N = cols, c.R = p.rows, c.weights_dtype = p.code;
        c.scale = (float)real(a[9]), c.layer = truth(a[10]), c.eps = real(a[11]);
        const bool b = a[3] != Py_None, pre = a[7] != Py_None;
        if (!b && (c.post || c.gate || a[13] != Py_None)) refuse(PyExc_ValueError, "post, gate and db go with b%s", "");
        if ((!c.post && c.post_bias) || (!pre && c.pre_bias) || pre != (a[2] != Py_None))
            refuse(PyExc_ValueError, "post_bias goes with post, dn and pre_bias with pre%s", "");
        if (pre && a[1] == Py_None) refuse(PyExc_ValueError, "y (x, where there is no b) is needed with pre%s", "");
        if (pre) c.y = address(tensor(a[1], "y"), type, rows, "y", device);
        void *stream = raw_stream(a[14], device);
        std::array<std::pair<const char *, at::Tensor>, 7> outs;
        int used = 0;
        auto rows_out = [&](PyObject *given, const char *name) {
            outs[used] = {name, output(given, rows, type, x, name, stream)};
            return address(outs[used++].second, type, rows, name, device);
        };
        auto sums_out = [&](const void *of, at::IntArrayRef shape, const char *name) -> float * {
            if (!of) return nullptr;
            outs[used] = {name, output(Py_None, shape, at::kFloat, x, name, stream)};
            return static_cast<float *>(outs[used++].second.data_ptr());
        };
        c.dx = rows_out(a[12], "dx");
        if (b) c.db = rows_out(a[13], "db");
        c.dgate = sums_out(c.gate, {c.R, cols}, "dgate");
        c.dpost = sums_out(c.post, {cols}, "dpost"), c.dpost_bias = sums_out(c.post_bias, {cols}, "dpost_bias");
        c.dpre = sums_out(c.pre, {cols}, "dpre"), c.dpre_bias = sums_out(c.pre_bias, {cols}, "dpre_bias");
        const size_t need = p_block_backward_ws(m, cols, c.R, c.dtype);
        at::Tensor ws;
        if (need) ws = scratch(need, x, stream);
        void *pw = need ? ws.data_ptr() : nullptr;
        int st = call([&] { return p_block_backward(&c, pw, need, stream); });
        if (st) return PyLong_FromLong(st);
        PyObject *d = PyDict_New();
        for (int i = 0; d && i < used; ++i) {
            PyObject *v = THPVariable_Wrap(outs[i].second);
            const int bad = !v || PyDict_SetItemString(d, outs[i].first, v);
            Py_XDECREF(v);
            if (bad) Py_CLEAR(d);
        }
        return d;
    });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(py_bind), nullptr},
                         {"address", FAST(py_address), nullptr},
                         {"stream", FAST(py_stream), nullptr},
                         {"gemm", FAST(py_gemm), nullptr},
                         {"route", FAST(py_route), nullptr},
                         {"route_backward", FAST(py_route_backward), nullptr},
                         {"moe", FAST(py_moe), nullptr},
                         {"linear", FAST(py_linear), nullptr},
                         {"layer", FAST(py_layer), nullptr},
                         {"block", FAST(py_block), nullptr},
                         {"block_backward", FAST(py_block_backward), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
