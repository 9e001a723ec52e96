// Argument marshalling of the norm and log-probability calls in compiled code: the checks of the Python binding on
// torch tensors, then the call through the C ABI.  A decode step makes these calls on a handful of rows, where reading
// a tensor's type, sizes, strides and address from Python takes longer than the kernel (4 x 2048 norm: 6.95 us a
// call from Python alone, 2.1 us from here).
//
// Every function returns 0 (done), a negative vh_status, or 1: the arguments are not of the usual kind (an output to
// be made, another stream, anything that does not fit), and the binding's own checks go on from there: they handle
// the call or say what is wrong with it.  Nothing is launched before all arguments have passed.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>

#include "../../include/verifyhead.h"

namespace {

// The entry points, bound by name to the library that the binding has loaded.
decltype(&vh_add_rmsnorm) p_add_rmsnorm;
decltype(&vh_add_rmsnorm_grad) p_add_rmsnorm_grad;
decltype(&vh_logits_logprobs) p_logits_logprobs;
decltype(&vh_logits_logprobs_grad) p_logits_logprobs_grad;
decltype(&vh_head_logprobs) p_head_logprobs;

struct Unusual {};  // thrown on the way out to "1"

const at::Tensor& tensor(PyObject* o) {
    if (!THPVariable_Check(o)) throw Unusual();
    return THPVariable_Unpack(o);
}

int row_type(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return VH_F32;
        case at::kBFloat16: return VH_BF16;
        case at::kHalf: return VH_F16;
        default: throw Unusual();
    }
}

struct Call {
    int dev;
    void* stream;

    // `first`: the call's first tensor, which must be on the current device.
    explicit Call(const at::Tensor& first) {
        if (!first.is_cuda()) throw Unusual();
        dev = first.get_device();
        if (dev != c10::cuda::current_device()) throw Unusual();
        stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    }
    void here(const at::Tensor& t) const {
        if (!t.is_cuda() || t.get_device() != dev || t.layout() != at::kStrided) throw Unusual();
    }
    // Address and row stride of a tensor [T][H] of that type with contiguous rows.
    void* rows(const at::Tensor& t, int64_t T, int64_t H, at::ScalarType type, int64_t* stride) const {
        here(t);
        if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != T || t.size(1) != H || (H > 1 && t.stride(1) != 1))
            throw Unusual();
        *stride = T > 1 ? t.stride(0) : (H > 1 ? H : 1);
        return t.data_ptr();
    }
    void* rows(PyObject* o, int64_t T, int64_t H, at::ScalarType type, int64_t* stride) const {
        *stride = 0;
        return o == Py_None ? nullptr : rows(tensor(o), T, H, type, stride);
    }
    void* vector(PyObject* o, int64_t n, at::ScalarType type) const {
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o);
        here(t);
        if (t.scalar_type() != type || t.numel() != n || !t.is_contiguous()) throw Unusual();
        return t.data_ptr();
    }
    // A norm's weight: of the rows' type or fp32.
    void* weight(PyObject* o, int64_t H, at::ScalarType type, int* f32) const {
        *f32 = o != Py_None && tensor(o).scalar_type() == at::kFloat;
        return vector(o, H, *f32 ? at::kFloat : type);
    }
    void* workspace(PyObject* o, size_t* bytes) const {
        *bytes = 0;
        if (o == Py_None) return nullptr;
        const at::Tensor& t = tensor(o);
        here(t);
        if (t.element_size() != 1 || !t.is_contiguous()) throw Unusual();
        *bytes = (size_t)t.numel();
        return t.data_ptr();
    }
};

int as_int(int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) throw Unusual();
    return (int)v;
}
float as_float(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unusual();
    }
    return (float)v;
}
int as_count(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        throw Unusual();
    }
    return as_int(v);
}

// The call itself, without the interpreter's lock: a launch may wait for room in the stream's queue, and a host function
// in that queue may want the lock.  The caller's arguments keep the tensors alive.
template <typename F, typename... A>
int launch(F f, A... a) {
    int st;
    Py_BEGIN_ALLOW_THREADS;
    st = f(a...);
    Py_END_ALLOW_THREADS;
    return st;
}

template <typename F>
PyObject* call(Py_ssize_t n, Py_ssize_t wanted, F f) {
    long st = 1;
    try {
        if (n == wanted) st = f();
    } catch (...) {  // Unusual, or torch's own refusal of a tensor without storage
        st = 1;
    }
    return PyLong_FromLong(st);
}

// x, residual, weight, eps, weight_offset, y, h, scales
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 8, [&]() -> int {
        const at::Tensor& x = tensor(a[0]);
        const Call c(x);
        if (x.dim() != 2 || a[5] == Py_None || (a[1] != Py_None && a[6] == Py_None)) throw Unusual();
        const at::ScalarType type = x.scalar_type();
        const int64_t T = x.size(0), H = x.size(1);
        const at::ScalarType out = tensor(a[5]).scalar_type();
        const int kind = a[7] == Py_None ? VH_NORM_SAME : out == at::kChar ? VH_NORM_INT8 : VH_NORM_E4M3;
        if (kind == VH_NORM_SAME ? out != type : (out != at::kChar && out != at::kFloat8_e4m3fn)) throw Unusual();
        int64_t xs, rs, ys, hs;
        int f32;
        void* xp = c.rows(x, T, H, type, &xs);
        void* rp = c.rows(a[1], T, H, type, &rs);
        void* wp = c.weight(a[2], H, type, &f32);
        void* yp = c.rows(a[5], T, H, out, &ys);
        void* hp = c.rows(a[6], T, H, type, &hs);
        float* sp = static_cast<float*>(c.vector(a[7], T, at::kFloat));
        return launch(p_add_rmsnorm, xp, rp, wp, row_type(type), f32, as_int(T), as_int(H), xs, rs, as_float(a[3]),
                      as_float(a[4]), yp, ys, kind, hp, hs, sp, c.stream);
    });
}

// dy, h, weight, eps, weight_offset, dh, dx, dweight, ws
PyObject* add_rmsnorm_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 9, [&]() -> int {
        const at::Tensor& h = tensor(a[1]);
        const Call c(h);
        if (h.dim() != 2 || a[6] == Py_None || (a[2] != Py_None) != (a[7] != Py_None) || (a[7] != Py_None && a[8] == Py_None))
            throw Unusual();
        const at::ScalarType type = h.scalar_type();
        const int64_t T = h.size(0), H = h.size(1);
        int64_t ys, hs, es, xs;
        int f32;
        size_t bytes;
        void* hp = c.rows(h, T, H, type, &hs);
        void* yp = c.rows(tensor(a[0]), T, H, type, &ys);
        void* wp = c.weight(a[2], H, type, &f32);
        void* ep = c.rows(a[5], T, H, type, &es);
        void* xp = c.rows(a[6], T, H, type, &xs);
        float* dw = static_cast<float*>(c.vector(a[7], H, at::kFloat));
        void* ws = c.workspace(a[8], &bytes);
        return launch(p_add_rmsnorm_grad, yp, hp, wp, ep, row_type(type), f32, as_int(T), as_int(H), ys, hs, es,
                      as_float(a[3]), as_float(a[4]), xp, xs, dw, ws, bytes, c.stream);
    });
}

// The outputs and the workspace of a log-probability call, all given, from a[0] on.
struct Outputs {
    float *logprob, *entropy, *lse, *top_logprobs;
    int32_t* top_ids;
    void* ws;
    size_t bytes;
    Outputs(const Call& c, PyObject* const* a, int64_t R, int n, bool tokens) {
        for (int i = 0; i < 6; ++i)
            if (a[i] == Py_None) throw Unusual();
        float* lp = static_cast<float*>(c.vector(a[0], R, at::kFloat));
        logprob = tokens ? lp : nullptr;
        entropy = static_cast<float*>(c.vector(a[1], R, at::kFloat));
        lse = static_cast<float*>(c.vector(a[2], R, at::kFloat));
        top_ids = n > 0 ? static_cast<int32_t*>(c.vector(a[3], R * n, at::kInt)) : nullptr;
        top_logprobs = n > 0 ? static_cast<float*>(c.vector(a[4], R * n, at::kFloat)) : nullptr;
        ws = c.workspace(a[5], &bytes);
    }
};

// logits, tokens, top_n, logprob, entropy, lse, top_ids, top_logprobs, ws
PyObject* logits_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 9, [&]() -> int {
        const at::Tensor& x = tensor(a[0]);
        const Call c(x);
        if (x.dim() != 2) throw Unusual();
        const int64_t R = x.size(0), V = x.size(1);
        const int top = as_count(a[2]);
        int64_t stride;
        void* xp = c.rows(x, R, V, x.scalar_type(), &stride);
        const int32_t* tp = static_cast<const int32_t*>(c.vector(a[1], R, at::kInt));
        const Outputs o(c, a + 3, R, top, tp != nullptr);
        return launch(p_logits_logprobs, xp, row_type(x.scalar_type()), as_int(R), as_int(V), stride, tp, top, o.logprob,
                      o.entropy, o.lse, o.top_ids, o.top_logprobs, o.ws, o.bytes, c.stream);
    });
}

// logits, tokens, lse, entropy, g_logprob, g_entropy, dlogits
PyObject* logits_logprobs_grad(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 7, [&]() -> int {
        const at::Tensor& x = tensor(a[0]);
        const Call c(x);
        if (x.dim() != 2 || a[6] == Py_None) throw Unusual();
        const int64_t R = x.size(0), V = x.size(1);
        int64_t xs, ds;
        void* xp = c.rows(x, R, V, x.scalar_type(), &xs);
        const int32_t* tp = static_cast<const int32_t*>(c.vector(a[1], R, at::kInt));
        const float* f[4];
        for (int i = 0; i < 4; ++i) f[i] = static_cast<const float*>(c.vector(a[2 + i], R, at::kFloat));
        void* dp = c.rows(a[6], R, V, x.scalar_type(), &ds);
        return launch(p_logits_logprobs_grad, xp, row_type(x.scalar_type()), as_int(R), as_int(V), xs, tp, f[0], f[1], f[2],
                      f[3], dp, ds, c.stream);
    });
}

// hidden, W_full, tokens, top_n, logprob, entropy, lse, top_ids, top_logprobs, ws
PyObject* head_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return call(n, 10, [&]() -> int {
        const at::Tensor& x = tensor(a[0]);
        const at::Tensor& w = tensor(a[1]);
        const Call c(x);
        c.here(x);
        c.here(w);
        if (x.dim() != 2 || w.dim() != 2 || x.size(1) != w.size(1) || !x.is_contiguous() || !w.is_contiguous() ||
            x.scalar_type() != at::kBFloat16 || w.scalar_type() != at::kBFloat16)
            throw Unusual();
        const int64_t R = x.size(0);
        const int top = as_count(a[3]);
        const int32_t* tp = static_cast<const int32_t*>(c.vector(a[2], R, at::kInt));
        const Outputs o(c, a + 4, R, top, tp != nullptr);
        return launch(p_head_logprobs, x.data_ptr(), w.data_ptr(), tp, as_int(R), as_int(x.size(1)), as_int(w.size(0)), top,
                      o.logprob, o.entropy, o.lse, o.top_ids, o.top_logprobs, o.ws, o.bytes, c.stream);
    });
}

// name, address
PyObject* bind(PyObject*, PyObject* args) {
    const char* name;
    unsigned long long at;
    if (!PyArg_ParseTuple(args, "sK", &name, &at)) return nullptr;
    void* p = reinterpret_cast<void*>(static_cast<uintptr_t>(at));
    if (!std::strcmp(name, "vh_add_rmsnorm"))
        p_add_rmsnorm = reinterpret_cast<decltype(p_add_rmsnorm)>(p);
    else if (!std::strcmp(name, "vh_add_rmsnorm_grad"))
        p_add_rmsnorm_grad = reinterpret_cast<decltype(p_add_rmsnorm_grad)>(p);
    else if (!std::strcmp(name, "vh_logits_logprobs"))
        p_logits_logprobs = reinterpret_cast<decltype(p_logits_logprobs)>(p);
    else if (!std::strcmp(name, "vh_logits_logprobs_grad"))
        p_logits_logprobs_grad = reinterpret_cast<decltype(p_logits_logprobs_grad)>(p);
    else if (!std::strcmp(name, "vh_head_logprobs"))
        p_head_logprobs = reinterpret_cast<decltype(p_head_logprobs)>(p);
    else
        return PyErr_Format(PyExc_ValueError, "no entry point %s", name);
    Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"add_rmsnorm", fast(add_rmsnorm), METH_FASTCALL, nullptr},
    {"add_rmsnorm_grad", fast(add_rmsnorm_grad), METH_FASTCALL, nullptr},
    {"logits_logprobs", fast(logits_logprobs), METH_FASTCALL, nullptr},
    {"logits_logprobs_grad", fast(logits_logprobs_grad), METH_FASTCALL, nullptr},
    {"head_logprobs", fast(head_logprobs), METH_FASTCALL, nullptr},
    {"bind", bind, METH_VARARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
