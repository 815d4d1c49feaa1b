// s6_torch.cpp -- the Python module _s6_torch: marshals the training-step calls
// from torch tensors to the C ABI of include/s6.h.
//
// At small sizes the time of a call is the time on the host: checks of eight
// tensors and four allocations took 17 to 40 us in Python beside kernels of 2 to
// 10 us, and take 4 to 8 us here.  The module holds no arithmetic and no state.
// Every function takes positional arguments from its wrapper in the package
// (which has the signature and the documentation), raises TypeError for a wrong
// type and ValueError for a wrong place, layout or shape, and returns the C
// ABI's negative status as an int for the wrapper to raise.
//
// Outputs and workspaces are allocated on the current stream of the tensors'
// device, which is also the stream of the launch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdio>
#include <string>
#include <vector>

#include "s6.h"

namespace {

// A Python exception that has been set.
struct Raised {};

template <typename... A>
[[noreturn]] void fail(PyObject *type, const char *fmt, A... args) {
    PyErr_Format(type, fmt, args...);
    throw Raised{};
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised{};
    return v != 0;
}

const char *type_name(at::ScalarType t) { return c10::toString(t); }

std::string shape_name(at::IntArrayRef shape) {
    std::string s = "(";
    for (size_t i = 0; i < shape.size(); ++i)
        s += (i ? ", " : "") + std::to_string(shape[i]);
    return s + (shape.size() == 1 ? ",)" : ")");
}

s6_stream_t stream_of(const at::Device &dev) {
    return reinterpret_cast<s6_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device &dev) {
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// A tensor argument: contiguous and on a CUDA device.
const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, "%s must be a torch.Tensor", name);
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda())
        fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
    if (!t.is_contiguous())
        fail(PyExc_ValueError, "%s must be contiguous", name);
    return t;
}

int code_of(const at::Tensor &t, const char *name) {
    if (t.scalar_type() == at::kFloat)
        return S6_F32;
    if (t.scalar_type() == at::kBFloat16)
        return S6_BF16;
    fail(PyExc_TypeError, "%s must be float32 or bfloat16, got %s", name, type_name(t.scalar_type()));
}

void check(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev) {
    if (t.device() != dev)
        fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
    if (t.scalar_type() != type)
        fail(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
    if (t.sizes() != shape) {
        fail(PyExc_ValueError, "%s has shape %s, expected %s", name, shape_name(t.sizes()).c_str(),
             shape_name(shape).c_str());
    }
}

// An optional tensor argument of a known type and shape: its address, or null for None.
void *pointer(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape, const at::Device &dev) {
    if (o == Py_None)
        return nullptr;
    const at::Tensor &t = tensor(o, name);
    check(t, name, type, shape, dev);
    return t.data_ptr();
}

void *address(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject *wrap(const at::Tensor &t) {
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *or_status(int status, std::initializer_list<PyObject *> items) {
    PyObject *out = status == S6_OK ? PyTuple_New(static_cast<Py_ssize_t>(items.size())) : nullptr;
    Py_ssize_t i = 0;
    bool whole = out != nullptr;
    for (PyObject *o : items) {
        whole = whole && o;
        if (out)
            PyTuple_SET_ITEM(out, i++, o);
        else
            Py_XDECREF(o);
    }
    if (status != S6_OK)
        return PyLong_FromLong(status);
    if (!whole)
        Py_CLEAR(out);
    return out;
}

at::Tensor workspace(int64_t bytes, const at::Device &dev) {
    if (bytes < 0)
        return at::Tensor();  // the call itself then returns the same status
    return empty({bytes}, at::kByte, dev);
}

// The C call, without the interpreter's lock: a launch may wait for room in a queue.
template <typename F>
int unlocked(F call) {
    PyThreadState *state = PyEval_SaveThread();
    const int st = call();
    PyEval_RestoreThread(state);
    return st;
}

// Every entry point runs in here: no C++ exception passes into Python.
template <typename F>
PyObject *guarded(Py_ssize_t nargs, Py_ssize_t want, F body) {
    if (nargs != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, nargs);
        return nullptr;
    }
    try {
        return body();
    } catch (const Raised &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

s6_norm_dims norm_dims(const at::Tensor &x, at::ScalarType branch, double eps, const char *name) {
    if (x.dim() < 1)
        fail(PyExc_ValueError, "x must have a last dimension to normalise");
    s6_norm_dims d;
    d.x_dtype = code_of(x, "x");
    if (branch != x.scalar_type() && branch != at::kBFloat16)
        fail(PyExc_TypeError, "%s must be %s, or bfloat16 beside a float32 x, got %s", name,
             type_name(x.scalar_type()), type_name(branch));
    d.y_dtype = branch == x.scalar_type() ? d.x_dtype : static_cast<int32_t>(S6_BF16);
    d.width = x.size(-1);
    d.rows = d.width ? x.numel() / d.width : 0;
    d.eps = static_cast<float>(eps);
    return d;
}

// (x, w, b, eps, r, s, y, y_dtype, want_stats) -> (y, s, mean, rstd)
PyObject *layernorm_fwd(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded(nargs, 9, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x");
        const double eps = PyFloat_AsDouble(a[3]);
        if (eps == -1.0 && PyErr_Occurred())
            throw Raised{};
        const bool want_stats = truth(a[8]);
        PyObject *po_r = a[4], *po_s = a[5], *po_y = a[6];
        at::ScalarType branch = x.scalar_type();
        if (a[7] != Py_None) {
            if (!THPDtype_Check(a[7]))
                fail(PyExc_TypeError, "y_dtype must be a torch.dtype");
            branch = reinterpret_cast<THPDtype *>(a[7])->scalar_type;
        } else if (po_r != Py_None) {
            branch = tensor(po_r, "r").scalar_type();
        } else if (po_y != Py_None) {
            branch = tensor(po_y, "y").scalar_type();
        }
        if (po_s != Py_None && po_r == Py_None)
            fail(PyExc_ValueError, "s is the sum x + r: it needs r");
        const s6_norm_dims dims = norm_dims(x, branch, eps, "the branch type");
        const at::Device dev = x.device();
        const at::IntArrayRef shape = x.sizes(), width = shape.slice(shape.size() - 1),
                              rows = shape.slice(0, shape.size() - 1);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        const void *r = pointer(po_r, "r", branch, shape, dev);
        const void *w = pointer(a[1], "w", at::kFloat, width, dev), *b = pointer(a[2], "b", at::kFloat, width, dev);
        void *s = pointer(po_s, "s", x.scalar_type(), shape, dev), *y = pointer(po_y, "y", branch, shape, dev);
        at::Tensor new_s, new_y, mean, rstd;
        if (po_y == Py_None)
            y = address(new_y = empty(shape, branch, dev));
        if (po_r != Py_None && po_s == Py_None)
            s = address(new_s = empty(shape, x.scalar_type(), dev));
        if (want_stats) {
            mean = empty(rows, at::kFloat, dev);
            rstd = empty(rows, at::kFloat, dev);
        }
        const s6_stream_t stream = stream_of(dev);
        const int st = unlocked([&] {
            return s6_layernorm_fwd(&dims, x.data_ptr(), r, static_cast<const float *>(w),
                                        static_cast<const float *>(b), s, y, static_cast<float *>(address(mean)),
                                        static_cast<float *>(address(rstd)), stream);
        });
        return or_status(st, {po_y == Py_None ? wrap(new_y) : Py_NewRef(po_y),
                              po_r == Py_None   ? Py_NewRef(a[0])
                              : po_s == Py_None ? wrap(new_s)
                                                : Py_NewRef(po_s),
                              wrap(mean), wrap(rstd)});
    });
}

// (dy, x, mean, rstd, w, ds, dx, want_params) -> (dx, dw, db)
PyObject *layernorm_bwd(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded(nargs, 8, [&]() -> PyObject * {
        const at::Tensor &dy = tensor(a[0], "dy"), &x = tensor(a[1], "x");
        const bool want_params = truth(a[7]);
        const s6_norm_dims dims = norm_dims(x, dy.scalar_type(), 0.0, "dy");
        const at::Device dev = x.device();
        const at::IntArrayRef shape = x.sizes(), width = shape.slice(shape.size() - 1),
                              rows = shape.slice(0, shape.size() - 1);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        check(dy, "dy", dy.scalar_type(), shape, dev);
        const at::Tensor &mean = tensor(a[2], "mean"), &rstd = tensor(a[3], "rstd");
        check(mean, "mean", at::kFloat, rows, dev);
        check(rstd, "rstd", at::kFloat, rows, dev);
        const void *w = pointer(a[4], "w", at::kFloat, width, dev), *ds = pointer(a[5], "ds", at::kFloat, shape, dev);
        at::Tensor new_dx, dw, db;
        void *dx = a[6] == Py_None ? address(new_dx = empty(shape, at::kFloat, dev))
                                   : pointer(a[6], "dx", at::kFloat, shape, dev);
        if (want_params) {
            dw = empty(width, at::kFloat, dev);
            db = empty(width, at::kFloat, dev);
        }
        const at::Tensor ws = workspace(s6_layernorm_bwd_workspace(&dims), dev);
        const s6_stream_t stream = stream_of(dev);
        const int st = unlocked([&] {
            return s6_layernorm_bwd(
            &dims, x.data_ptr(), static_cast<const float *>(mean.data_ptr()),
            static_cast<const float *>(rstd.data_ptr()), static_cast<const float *>(w), dy.data_ptr(),
            static_cast<const float *>(ds), static_cast<float *>(dx), static_cast<float *>(address(dw)),
            static_cast<float *>(address(db)), address(ws), ws.defined() ? ws.numel() : 0, stream);
        });
        return or_status(st, {a[6] == Py_None ? wrap(new_dx) : Py_NewRef(a[6]), wrap(dw), wrap(db)});
    });
}

// (x, conv_w, dout, conv_b) -> (dx, dconv_w, dconv_b)
PyObject *conv_bwd(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded(nargs, 4, [&]() -> PyObject * {
        const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "conv_w"), &g = tensor(a[2], "dout");
        if (x.dim() != 3)
            fail(PyExc_ValueError, "x must be [batch, seqlen, d_inner]");
        if (w.dim() != 2)
            fail(PyExc_ValueError, "conv_w must be [d_inner, width]");
        const int io = code_of(x, "x");
        if (g.scalar_type() != at::kFloat && g.scalar_type() != x.scalar_type())
            fail(PyExc_TypeError, "dout must be float32 or %s, got %s", type_name(x.scalar_type()),
                 type_name(g.scalar_type()));
        const at::Device dev = x.device();
        const int64_t d = x.size(2), K = w.size(1);
        const c10::cuda::OptionalCUDAGuard guard(dev);
        check(w, "conv_w", at::kFloat, {d, K}, dev);
        check(g, "dout", g.scalar_type(), x.sizes(), dev);
        const void *b = pointer(a[3], "conv_b", at::kFloat, {d}, dev);
        const s6_dims dims{x.size(0), x.size(1), d, 1, K, io};
        const at::Tensor dx = empty(x.sizes(), at::kFloat, dev), dw = empty({d, K}, at::kFloat, dev);
        const at::Tensor db = a[3] == Py_None ? at::Tensor() : empty({d}, at::kFloat, dev);
        const at::Tensor ws = workspace(causal_conv1d_silu_bwd_workspace(&dims), dev);
        const s6_stream_t stream = stream_of(dev);
        const int st = unlocked([&] {
            return causal_conv1d_silu_bwd(
            &dims, x.data_ptr(), static_cast<const float *>(w.data_ptr()), static_cast<const float *>(b), g.data_ptr(),
            code_of(g, "dout"), static_cast<float *>(dx.data_ptr()), static_cast<float *>(dw.data_ptr()),
            static_cast<float *>(address(db)), address(ws), ws.defined() ? ws.numel() : 0, stream);
        });
        return or_status(st, {wrap(dx), wrap(dw), wrap(db)});
    });
}

// The tensors of a gradient call as the host arrays that the library reads.
struct GradList {
    std::vector<void *> ptr;
    std::vector<int64_t> numel;
    std::vector<int32_t> type;
    at::Device dev = at::Device(at::kCUDA, 0);
    int64_t count() const { return static_cast<int64_t>(ptr.size()); }

    // grads: a list; None entries are left out.  The device is that of norm, or of the
    // first tensor, or the current one.
    GradList(PyObject *grads, PyObject *norm) {
        if (!PyList_Check(grads))
            fail(PyExc_TypeError, "grads must be a list");
        const Py_ssize_t n = PyList_GET_SIZE(grads);
        ptr.reserve(n);
        numel.reserve(n);
        type.reserve(n);
        bool placed = norm != Py_None;
        if (placed) {
            const at::Tensor &t = tensor(norm, "norm");
            if (t.scalar_type() != at::kFloat || t.numel() != 1)
                fail(PyExc_ValueError, "norm must be a float32 tensor of 1 element");
            dev = t.device();
        }
        for (Py_ssize_t i = 0; i < n; ++i) {
            PyObject *o = PyList_GET_ITEM(grads, i);
            if (o == Py_None)
                continue;
            char name[32];
            std::snprintf(name, sizeof(name), "grads[%zd]", i);
            const at::Tensor &t = tensor(o, name);
            if (!placed) {
                dev = t.device();
                placed = true;
            }
            if (t.device() != dev)
                fail(PyExc_ValueError, "%s is on %s, expected %s", name, t.device().str().c_str(), dev.str().c_str());
            type.push_back(code_of(t, name));
            ptr.push_back(t.data_ptr());
            numel.push_back(t.numel());
        }
        if (!placed)
            dev = at::Device(at::kCUDA, c10::cuda::current_device());
    }
};

// (grads, norm) -> (norm,)
PyObject *grad_norm(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded(nargs, 2, [&]() -> PyObject * {
        const GradList g(a[0], a[1]);
        const c10::cuda::OptionalCUDAGuard guard(g.dev);
        at::Tensor norm = a[1] == Py_None ? empty({}, at::kFloat, g.dev) : THPVariable_Unpack(a[1]);
        const at::Tensor ws = workspace(s6_grad_workspace(g.count(), g.numel.data()), g.dev);
        const s6_stream_t stream = stream_of(g.dev);
        const int st = unlocked([&] {
            return s6_grad_norm(g.count(), g.ptr.data(), g.numel.data(), g.type.data(),
                                    static_cast<float *>(norm.data_ptr()), address(ws), ws.defined() ? ws.numel() : 0,
                                    stream);
        });
        return or_status(st, {a[1] == Py_None ? wrap(norm) : Py_NewRef(a[1])});
    });
}

// (grads, norm, max_norm, eps) -> ()
PyObject *grad_clip(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded(nargs, 4, [&]() -> PyObject * {
        const at::Tensor &norm = tensor(a[1], "norm");
        const GradList g(a[0], a[1]);
        const c10::cuda::OptionalCUDAGuard guard(g.dev);
        const float max_norm = static_cast<float>(PyFloat_AsDouble(a[2])), eps = static_cast<float>(PyFloat_AsDouble(a[3]));
        if (PyErr_Occurred())
            throw Raised{};
        const s6_stream_t stream = stream_of(g.dev);
        const int st = unlocked([&] {
            return s6_grad_clip(g.count(), g.ptr.data(), g.numel.data(), g.type.data(),
                                    static_cast<const float *>(norm.data_ptr()), max_norm, eps, stream);
        });
        return or_status(st, {});
    });
}

// (grads, max_norm, eps, norm) -> (norm,)
PyObject *clip_grad_norm(PyObject *, PyObject *const *a, Py_ssize_t nargs) {
    return guarded(nargs, 4, [&]() -> PyObject * {
        const GradList g(a[0], a[3]);
        const c10::cuda::OptionalCUDAGuard guard(g.dev);
        const float max_norm = static_cast<float>(PyFloat_AsDouble(a[1])), eps = static_cast<float>(PyFloat_AsDouble(a[2]));
        if (PyErr_Occurred())
            throw Raised{};
        at::Tensor norm = a[3] == Py_None ? empty({}, at::kFloat, g.dev) : THPVariable_Unpack(a[3]);
        const at::Tensor ws = workspace(s6_grad_workspace(g.count(), g.numel.data()), g.dev);
        const s6_stream_t stream = stream_of(g.dev);
        const int st = unlocked([&] {
            return s6_clip_grad_norm(g.count(), g.ptr.data(), g.numel.data(), g.type.data(), max_norm, eps,
                                         static_cast<float *>(norm.data_ptr()), address(ws),
                                         ws.defined() ? ws.numel() : 0, stream);
        });
        return or_status(st, {a[3] == Py_None ? wrap(norm) : Py_NewRef(a[3])});
    });
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<layernorm_fwd>("layernorm_fwd"), method<layernorm_bwd>("layernorm_bwd"),
                         method<conv_bwd>("conv_bwd"),           method<grad_norm>("grad_norm"),
                         method<grad_clip>("grad_clip"),         method<clip_grad_norm>("clip_grad_norm"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_s6_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__s6_torch(void) { return PyModule_Create(&module); }
