// Python calls of the 4-bit weights and the mixture-of-experts operators.
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

#include "../../include/libtq2_moe.h"

namespace {

decltype(&q4_gemm_workspace_size) p_gemm_ws;
decltype(&q4_gemm) p_gemm;
decltype(&moe_route) p_route;
decltype(&moe_route_backward) p_route_backward;
decltype(&q4_moe_workspace_size) p_moe_ws;
decltype(&q4_moe) p_moe;

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
        count(n, 6);
        auto at = [&](int i) { return PyLong_AsVoidPtr(a[i]); };
        p_gemm_ws = reinterpret_cast<decltype(p_gemm_ws)>(at(0));
        p_gemm = reinterpret_cast<decltype(p_gemm)>(at(1));
        p_route = reinterpret_cast<decltype(p_route)>(at(2));
        p_route_backward = reinterpret_cast<decltype(p_route_backward)>(at(3));
        p_moe_ws = reinterpret_cast<decltype(p_moe_ws)>(at(4));
        p_moe = reinterpret_cast<decltype(p_moe)>(at(5));
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

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(py_bind), nullptr},
                         {"address", FAST(py_address), nullptr},
                         {"stream", FAST(py_stream), nullptr},
                         {"gemm", FAST(py_gemm), nullptr},
                         {"route", FAST(py_route), nullptr},
                         {"route_backward", FAST(py_route_backward), nullptr},
                         {"moe", FAST(py_moe), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
