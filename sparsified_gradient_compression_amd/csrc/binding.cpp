// binding.cpp -- the checks and argument blocks of the layer and gradient-set
// operators for torch tensors, as a CPython module over the C ABI.
//
// A call of the smallest sizes takes a few microseconds on the GPU, and a
// gradient set has hundreds of tensors: read through Python's attributes,
// their types, shapes and addresses would take longer than the kernels
// (161 gradients and outputs: 70 us there, 4 us here).
#include <c10/core/GradMode.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>
#include <vector>

#include "dgc.h"

namespace {

// Raised as ValueError by the entry points below.
struct Refusal {
    std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refusal{what}; }

const at::Tensor& unpacked(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor");
    return THPVariable_Unpack(o);
}

const at::Tensor* tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = unpacked(o, name);
    // what these calls write has no history, as of torch's own calls with out=
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(std::string(name) + ": requires a gradient, and these calls record none: call them under torch.no_grad()");
    return &t;
}

// Tensors that a call has written: what saved one of them for a backward pass finds out.
void wrote(std::initializer_list<const at::Tensor*> outs) {
    for (const at::Tensor* t : outs)
        if (t && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

int done(int rc, std::initializer_list<const at::Tensor*> outs) {
    if (rc == DGC_OK) wrote(outs);
    return rc;
}

const at::Tensor& needed(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) refuse(std::string(name) + ": expected a tensor");
    return *t;
}

int64_t type_code(at::ScalarType t) {
    return t == at::kBFloat16 ? DGC_BF16 : t == at::kHalf ? DGC_FP16 : t == at::kFloat ? DGC_FP32 : 0;
}

std::string shape(const at::Tensor& t) {
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + ")";
}

// What the tensors of one call share.
struct Call {
    const char* fn;
    at::ScalarType type;
    int device;

    Call(const char* name, const at::Tensor& x) : fn(name), type(x.scalar_type()), device(x.get_device()) {
        if (type != at::kBFloat16 && type != at::kHalf)
            refuse(std::string(fn) + ": expected bfloat16 or float16, got " + c10::toString(type));
    }

    void place(const at::Tensor& t, const char* name, at::ScalarType want) const {
        if (t.scalar_type() != want)
            refuse(std::string(name) + ": expected " + c10::toString(want) + ", got " + c10::toString(t.scalar_type()));
        if (!t.is_cuda() || t.get_device() != device)
            refuse(std::string(name) + ": expected a tensor on the device of x, a GPU");
    }

    template <class P>
    void mat(const at::Tensor* t, const char* name, int64_t rows, int64_t cols, at::ScalarType want, P& p,
             int64_t& ld) const {
        p = nullptr;
        ld = 0;
        if (!t) return;
        place(*t, name, want);
        if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols)
            refuse(std::string(name) + ": expected shape (" + std::to_string(rows) + ", " + std::to_string(cols) +
                   "), got " + shape(*t));
        ld = rows > 1 ? t->stride(0) : cols;
        if ((t->stride(1) != 1 && cols > 1) || ld < cols)
            refuse(std::string(name) + ": columns must be contiguous and rows must not overlap");
        p = t->data_ptr();
    }

    template <class P>
    void vec(const at::Tensor* t, const char* name, int64_t n, at::ScalarType want, P& p) const {
        p = nullptr;
        if (!t) return;
        place(*t, name, want);
        if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
            refuse(std::string(name) + ": expected " + std::to_string(n) + " contiguous elements");
        p = t->data_ptr();
    }

    // m, n, k of x [m, k] and w [n, k]
    void sizes(const at::Tensor& x, const at::Tensor& w, int64_t& m, int64_t& n, int64_t& k) const {
        if (x.dim() != 2 || w.dim() != 2 || x.size(1) != w.size(1))
            refuse(std::string(fn) + ": x and its weight must be matrices of equal width, got " + shape(x) + " and " +
                   shape(w));
        m = x.size(0);
        n = w.size(0);
        k = x.size(1);
    }

    void space(const at::Tensor* w, void*& p, size_t& bytes) const {
        p = nullptr;
        bytes = 0;
        if (!w) return;
        if (!w->is_cuda() || w->get_device() != device || !w->is_contiguous())
            refuse("workspace: expected a contiguous tensor on the device of x");
        bytes = w->nbytes();
        p = bytes ? w->data_ptr() : nullptr;
    }

    // The type of weight gradients: x's, or binary32.
    at::ScalarType gradients(const at::Tensor* a, const at::Tensor* b) const {
        const at::ScalarType g = a ? a->scalar_type() : b ? b->scalar_type() : type;
        if (g != type && g != at::kFloat)
            refuse(std::string(fn) + ": weight gradients are of x's type or float32, not " + c10::toString(g));
        return g;
    }
};

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse("expected an integer");
    }
    return v;
}

hipStream_t stream_of(PyObject* o) { return reinterpret_cast<hipStream_t>(uintptr_t(integer(o))); }

// Runs f, which returns a DGC_* code; refusals become ValueError.
template <class F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F f) {
    if (have != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Refusal& r) {
        PyErr_SetString(PyExc_ValueError, r.what.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// linear(act, x, w, bias, residual, y, pre, workspace, stream)
PyObject* py_linear(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 9, [&] {
        const at::Tensor &x = needed(o[1], "x"), &w = needed(o[2], "w");
        const Call c("linear", x);
        dgc_linear_args a{};
        a.type = type_code(c.type);
        a.act = integer(o[0]);
        c.sizes(x, w, a.m, a.n, a.k);
        c.mat(&x, "x", a.m, a.k, c.type, a.x, a.ldx);
        c.mat(&w, "w", a.n, a.k, c.type, a.w, a.ldw);
        c.vec(tensor(o[3], "bias"), "bias", a.n, c.type, a.bias);
        c.mat(tensor(o[4], "residual"), "residual", a.m, a.n, c.type, a.residual, a.ldr);
        const at::Tensor *y = &needed(o[5], "out"), *pre = tensor(o[6], "pre");
        c.mat(y, "out", a.m, a.n, c.type, a.y, a.ldy);
        c.mat(pre, "pre", a.m, a.n, c.type, a.pre, a.ldpre);
        void* ws;
        size_t bytes;
        c.space(tensor(o[7], "workspace"), ws, bytes);
        return done(dgc_linear(&a, ws, bytes, stream_of(o[8])), {y, pre});
    });
}

// linear_backward(act, dy, x, w, pre, dx, dw, dbias, workspace, stream)
PyObject* py_linear_backward(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 10, [&] {
        const at::Tensor &x = needed(o[2], "x"), &w = needed(o[3], "w");
        const at::Tensor *pre = tensor(o[4], "pre"), *dx = tensor(o[5], "dx"), *dw = tensor(o[6], "dw");
        const at::Tensor* db = tensor(o[7], "dbias");
        const Call c("linear_backward", x);
        const at::ScalarType g = c.gradients(dw, db);
        dgc_linear_backward_args a{};
        a.type = type_code(c.type);
        a.grad_type = type_code(g);
        a.act = integer(o[0]);
        if ((a.act & ~int64_t(DGC_DZ_ROUNDED)) != DGC_ACT_NONE && !pre) refuse("linear_backward: an activation's gradient needs pre");
        c.sizes(x, w, a.m, a.n, a.k);
        c.mat(&needed(o[1], "dy"), "dy", a.m, a.n, c.type, a.dy, a.lddy);
        c.mat(&x, "x", a.m, a.k, c.type, a.x, a.ldx);
        c.mat(&w, "w", a.n, a.k, c.type, a.w, a.ldw);
        c.mat(pre, "pre", a.m, a.n, c.type, a.pre, a.ldpre);
        c.mat(dx, "dx", a.m, a.k, c.type, a.dx, a.lddx);
        c.mat(dw, "dw", a.n, a.k, g, a.dw, a.lddw);
        c.vec(db, "dbias", a.n, g, a.dbias);
        void* ws;
        size_t bytes;
        c.space(tensor(o[8], "workspace"), ws, bytes);
        return done(dgc_linear_backward(&a, ws, bytes, stream_of(o[9])), {dx, dw, db});
    });
}

// gated_ffn(act, x, w_gate, w_up, h, gate, up, workspace, stream)
PyObject* py_gated_ffn(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 9, [&] {
        const at::Tensor &x = needed(o[1], "x"), &w = needed(o[2], "w_gate");
        const Call c("gated_ffn", x);
        dgc_gated_ffn_args a{};
        a.type = type_code(c.type);
        a.act = integer(o[0]);
        c.sizes(x, w, a.m, a.f, a.d);
        c.mat(&x, "x", a.m, a.d, c.type, a.x, a.ldx);
        c.mat(&w, "w_gate", a.f, a.d, c.type, a.w_gate, a.ldw_gate);
        c.mat(&needed(o[3], "w_up"), "w_up", a.f, a.d, c.type, a.w_up, a.ldw_up);
        const at::Tensor *h = &needed(o[4], "out"), *gate = tensor(o[5], "gate"), *up = tensor(o[6], "up");
        c.mat(h, "out", a.m, a.f, c.type, a.h, a.ldh);
        c.mat(gate, "gate", a.m, a.f, c.type, a.gate, a.ldgate);
        c.mat(up, "up", a.m, a.f, c.type, a.up, a.ldup);
        void* ws;
        size_t bytes;
        c.space(tensor(o[7], "workspace"), ws, bytes);
        return done(dgc_gated_ffn(&a, ws, bytes, stream_of(o[8])), {h, gate, up});
    });
}

// gated_ffn_backward(act, dh, x, w_gate, w_up, gate, up, dx, dw_gate, dw_up, workspace, stream)
PyObject* py_gated_ffn_backward(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 12, [&] {
        const at::Tensor &x = needed(o[2], "x"), &w = needed(o[3], "w_gate");
        const at::Tensor *dx = tensor(o[7], "dx"), *dg = tensor(o[8], "dw_gate"), *du = tensor(o[9], "dw_up");
        const Call c("gated_ffn_backward", x);
        if (!dg != !du) refuse("gated_ffn_backward: dw_gate and dw_up come together");
        const at::ScalarType g = c.gradients(dg, nullptr);
        dgc_gated_ffn_backward_args a{};
        a.type = type_code(c.type);
        a.grad_type = type_code(g);
        a.act = integer(o[0]);
        c.sizes(x, w, a.m, a.f, a.d);
        c.mat(&needed(o[1], "dh"), "dh", a.m, a.f, c.type, a.dh, a.lddh);
        c.mat(&x, "x", a.m, a.d, c.type, a.x, a.ldx);
        c.mat(&w, "w_gate", a.f, a.d, c.type, a.w_gate, a.ldw_gate);
        c.mat(&needed(o[4], "w_up"), "w_up", a.f, a.d, c.type, a.w_up, a.ldw_up);
        c.mat(&needed(o[5], "gate"), "gate", a.m, a.f, c.type, a.gate, a.ldgate);
        c.mat(&needed(o[6], "up"), "up", a.m, a.f, c.type, a.up, a.ldup);
        c.mat(dx, "dx", a.m, a.d, c.type, a.dx, a.lddx);
        c.mat(dg, "dw_gate", a.f, a.d, g, a.dw_gate, a.lddw_gate);
        c.mat(du, "dw_up", a.f, a.d, g, a.dw_up, a.lddw_up);
        void* ws;
        size_t bytes;
        c.space(tensor(o[10], "workspace"), ws, bytes);
        return done(dgc_gated_ffn_backward(&a, ws, bytes, stream_of(o[11])), {dx, dg, du});
    });
}

// A sequence of tensors, kept until the call that takes their addresses has returned.
struct Tensors {
    PyObject* fast = nullptr;
    std::vector<void*> data;

    Tensors() = default;
    Tensors(const Tensors&) = delete;
    ~Tensors() { Py_XDECREF(fast); }

    void wrote_all() const {
        for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(fast); ++i)
            wrote({&THPVariable_Unpack(PySequence_Fast_GET_ITEM(fast, i))});
    }
};

// A set's layout as the binding holds it: element counts and types, in bytes
// objects of int64 and int32.
struct Layout {
    const int64_t* sizes;
    const int32_t* types;
    Py_ssize_t count;
    int device;

    Layout(PyObject* s, PyObject* t, PyObject* d) : device(int(integer(d))) {
        if (!PyBytes_Check(s) || !PyBytes_Check(t)) refuse("expected the set's layout");
        count = PyBytes_GET_SIZE(s) / 8;
        if (PyBytes_GET_SIZE(t) != count * 4) refuse("expected the set's layout");
        sizes = reinterpret_cast<const int64_t*>(PyBytes_AS_STRING(s));
        types = reinterpret_cast<const int32_t*>(PyBytes_AS_STRING(t));
    }

    // out: what the call writes and does not read.  (Whether it requires a gradient is not looked up: of 161 views
    // that takes 6 us before the first launch, and that they were written is noted behind the last one.)
    void read(PyObject* seq, const char* what, Tensors& to, bool out = false) const {
        to.fast = PySequence_Fast(seq, "expected a sequence of tensors");
        if (!to.fast) {
            PyErr_Clear();
            refuse(std::string(what) + ": expected a sequence of tensors");
        }
        if (PySequence_Fast_GET_SIZE(to.fast) != count)
            refuse(std::string(what) + ": expected " + std::to_string(count) + " tensors");
        to.data.reserve(size_t(count));
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject* const item = PySequence_Fast_GET_ITEM(to.fast, i);
            const at::Tensor& t = out ? unpacked(item, what) : needed(item, what);
            if (t.numel() != sizes[i] || type_code(t.scalar_type()) != types[i])
                refuse(std::string(what) + ": tensor " + std::to_string(i) +
                       " differs from the set's shapes or dtypes");
            if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
                refuse(std::string(what) + ": expected contiguous tensors on the set's device");
            to.data.push_back(t.data_ptr());
        }
    }
};

double number(PyObject* o, const char* name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + ": expected a number");
    }
    return v;
}

// set_norm(set, sizes, types, device, grads, norm, unscale, out_norm, stream)
PyObject* py_set_norm(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 9, [&] {
        const Layout l(o[1], o[2], o[3]);
        Tensors g;
        l.read(o[4], "grads", g);
        const at::Tensor& total = needed(o[7], "total");
        return done(dgc_gradset_norm(reinterpret_cast<dgc_gradset*>(uintptr_t(integer(o[0]))), g.data.data(),
                                     int32_t(integer(o[5])), number(o[6], "unscale"),
                                     static_cast<double*>(total.data_ptr()), stream_of(o[8])),
                    {&total});
    });
}

// set_clip(set, sizes, types, device, grads, outs or None, clip, norm, unscale, out_norm, out_scale, stream)
PyObject* py_set_clip(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 12, [&] {
        const Layout l(o[1], o[2], o[3]);
        Tensors g, other;
        l.read(o[4], "grads", g);
        if (o[5] != Py_None) l.read(o[5], "out", other, true);
        const Tensors& out = o[5] == Py_None ? g : other;
        const at::Tensor &total = needed(o[9], "total"), &scale = needed(o[10], "scale");
        const int rc = dgc_gradset_clip(reinterpret_cast<dgc_gradset*>(uintptr_t(integer(o[0]))), g.data.data(),
                                        out.data.data(), number(o[6], "clip"),
                                        int32_t(integer(o[7])), number(o[8], "unscale"),
                                        static_cast<double*>(total.data_ptr()),
                                        static_cast<float*>(scale.data_ptr()), stream_of(o[11]));
        if (rc == DGC_OK) out.wrote_all();
        return done(rc, {&total, &scale});
    });
}

// set_pack(set, sizes, types, device, grads, flat, clip, norm, unscale, out_norm, out_scale, stream)
PyObject* py_set_pack(PyObject*, PyObject* const* o, Py_ssize_t count) {
    return guarded(count, 12, [&] {
        const Layout l(o[1], o[2], o[3]);
        Tensors g;
        l.read(o[4], "grads", g);
        const at::Tensor& flat = needed(o[5], "flat");
        int64_t n = 0;
        for (Py_ssize_t i = 0; i < l.count; ++i) n += l.sizes[i];
        if (flat.scalar_type() != at::kFloat || flat.numel() < n || !flat.is_cuda() ||
            flat.get_device() != l.device || !flat.is_contiguous())
            refuse("flat: expected at least " + std::to_string(n) +
                   " contiguous float32 elements on the set's device");
        const at::Tensor &total = needed(o[9], "total"), &scale = needed(o[10], "scale");
        return done(dgc_gradset_pack(reinterpret_cast<dgc_gradset*>(uintptr_t(integer(o[0]))), g.data.data(),
                                     static_cast<float*>(flat.data_ptr()), number(o[6], "clip"),
                                     int32_t(integer(o[7])), number(o[8], "unscale"),
                                     static_cast<double*>(total.data_ptr()), static_cast<float*>(scale.data_ptr()),
                                     stream_of(o[11])),
                    {&flat, &total, &scale});
    });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<py_linear>("linear"),
                         method<py_linear_backward>("linear_backward"),
                         method<py_gated_ffn>("gated_ffn"),
                         method<py_gated_ffn_backward>("gated_ffn_backward"),
                         method<py_set_norm>("set_norm"),
                         method<py_set_clip>("set_clip"),
                         method<py_set_pack>("set_pack"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dgc_torch", "libdgc's layer and gradient-set calls for torch tensors.",
                      -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dgc_torch() { return PyModule_Create(&module); }
