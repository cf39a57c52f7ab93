// Torch binding of wino_group_norm and wino_matmul (argument marshalling only): checks the tensors, makes the
// output, fills the ABI's structs and calls the library on the current stream.  A kernel can take less time than
// the dozens of Python statements this replaces.  The library's entry points are handed over by set_entries, so the
// module works with either of its builds.
//
// Each function returns the output tensor, or the library's status code when it refuses the call; tensors that do
// not fit together raise ValueError here.
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/utils/object_ptr.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/core/InferenceMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdio>
#include <stdexcept>
#include <string>

#include "../../include/wino.h"

namespace {

using Status = int (*)(const void*, void*);
struct Entries {
    Status group_norm = nullptr, matmul = nullptr;
} g_entries[2];   // release, debug

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

int code_of(at::ScalarType t) { return t == at::kBFloat16 ? WINO_BF16 : (t == at::kFloat ? WINO_F32 : -1); }

const at::Tensor* tensor(PyObject* o, const char* name) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return &THPVariable_Unpack(o);
}
const at::Tensor& required(PyObject* o, const char* name) {
    const at::Tensor* t = tensor(o, name);
    if (!t) refuse(std::string(name) + " must be a tensor");
    return *t;
}

void on(const char* name, const at::Tensor& t, const at::Tensor& first, at::ScalarType dtype) {
    if (t.device() != first.device()) refuse(std::string(name) + " is on " + t.device().str() + ", not on " + first.device().str());
    if (t.scalar_type() != dtype) refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + ", not " + c10::toString(dtype));
}

// The address of a contiguous fp32 parameter of the given shape; null for None.
const float* param(const char* name, const at::Tensor* t, const at::Tensor& first, at::IntArrayRef shape) {
    if (!t) return nullptr;
    on(name, *t, first, at::kFloat);
    if (t->sizes() != shape || !t->is_contiguous()) refuse(std::string(name) + " must be contiguous, one value per channel");
    return static_cast<const float*>(t->data_ptr());
}

// Elements between consecutive rows (the last dimension's vectors) of t, whose leading dimensions must collapse
// into one.
int64_t pitch_of(const char* name, const at::Tensor& t) {
    const auto sizes = t.sizes(), strides = t.strides();
    const int64_t last = sizes[sizes.size() - 1];
    if (t.is_contiguous()) return last;
    if (strides[sizes.size() - 1] != 1 && last != 1) refuse(std::string(name) + ": the last dimension must be contiguous");
    int64_t pitch = 0, rows = 1;   // of the dimensions seen so far, innermost first
    for (int64_t i = (int64_t)sizes.size() - 2; i >= 0; --i) {
        if (sizes[i] == 1) continue;
        if (rows == 1) pitch = strides[i];
        else if (strides[i] != pitch * rows) refuse(std::string(name) + ": rows must be evenly spaced");
        rows *= sizes[i];
    }
    return rows > 1 ? pitch : last;
}

// What torch keeps beside a tensor's memory and these operators do not look at is refused, not dropped: the sign of a
// lazily negated view, and gradients and forward-mode tangents (the operators have no derivatives).
template <typename... T>
void plain(const T*... t) {
    for (const at::Tensor* x : {t...}) {
        if (!x) continue;
        if (x->is_neg()) refuse("a tensor is a lazily negated view (as the imaginary part of a conjugate is): call resolve_neg() first");
        if (!x->unsafeGetTensorImpl()->autograd_meta()) continue;   // (most tensors: the rest takes library calls)
        if (c10::GradMode::is_enabled() && x->requires_grad())
            refuse("an input requires grad, and this operator has no backward pass: call it under torch.no_grad()");
        if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && x->_fw_grad(/*level=*/0).defined())
            refuse("an input carries a forward-mode tangent, and this operator has no derivative: unpack the dual tensor first");
    }
}

int as_int(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be an integer");
    }
    return v < -2147483647L || v > 2147483647L ? -1 : (int)v;
}
int size32(int64_t v) { return v > 2147483647 ? -1 : (int)v; }   // (the library refuses -1)

at::ScalarType dtype_or(PyObject* o, at::ScalarType otherwise) {
    if (o == Py_None) return otherwise;
    if (!THPDtype_Check(o)) refuse("out_dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// (at::empty without its dispatch)
at::Tensor new_tensor(at::IntArrayRef shape, at::ScalarType dtype, const at::Tensor& like) {
    return at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt);
}

template <typename F>
PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (const std::invalid_argument& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError& e) {
        THPObjectPtr torch(PyImport_ImportModule("torch"));
        THPObjectPtr type(torch ? PyObject_GetAttrString(torch.get(), "OutOfMemoryError") : nullptr);
        if (type) PyErr_SetString(type.get(), e.what_without_backtrace());
    } catch (const c10::Error& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

template <typename Args>
PyObject* run(Status fn, const Args& args, const at::Tensor& out, PyObject* given) {
    TORCH_CHECK(given == Py_None || !out.is_inference() || c10::InferenceMode::is_enabled(),
                "out is an inference tensor, which may only be written in inference mode");
    const int rc = fn(&args, c10::cuda::getCurrentCUDAStream(out.get_device()).stream());
    if (rc != WINO_OK) return PyLong_FromLong(rc);
    if (given != Py_None) {
        // (a graph that saved the given tensor for its backward pass finds out, as after torch's own in-place calls)
        out.unsafeGetTensorImpl()->bump_version();
        Py_INCREF(given);
        return given;
    }
    return THPVariable_Wrap(out);
}

// group_norm(x, groups, gamma, beta, eps, act, add, x2, out, out_dtype, debug)
PyObject* group_norm(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 11) refuse("group_norm takes 11 arguments");
        const at::Tensor& x = required(o[0], "x");
        const at::Tensor *gamma = tensor(o[2], "gamma"), *beta = tensor(o[3], "beta"), *add = tensor(o[6], "add"),
                         *x2 = tensor(o[7], "x2"), *given = tensor(o[8], "out");
        if (!x.is_cuda() || x.dim() != 4) refuse("x must be a CUDA tensor [N][H][W][C]");
        const at::ScalarType dtype = x.scalar_type();
        if (code_of(dtype) < 0) refuse(std::string("unsupported dtype ") + c10::toString(dtype));
        plain(&x, x2, add, gamma, beta, given);
        const auto sz = x.sizes();
        wino_group_norm_args g = {};
        int64_t C = sz[3];
        if (x2) {
            if (x2->dim() != 4 || x2->sizes().slice(0, 3) != sz.slice(0, 3)) refuse("x2 must be [N][H][W][C2] with x's N, H, W");
            on("x2", *x2, x, dtype);
            g.x2 = x2->data_ptr();
            g.x2_pitch = pitch_of("x2", *x2);
            g.C2 = size32(x2->size(3));
            C += x2->size(3);
        }
        const int64_t shape[4] = {sz[0], sz[1], sz[2], C}, per_image[2] = {sz[0], C}, per_channel[1] = {C};
        g.add = param("add", add, x, per_image);
        g.gamma = param("gamma", gamma, x, per_channel);
        g.beta = param("beta", beta, x, per_channel);
        const at::ScalarType odtype = given ? given->scalar_type() : dtype_or(o[9], dtype);
        if (code_of(odtype) < 0) refuse(std::string("unsupported output dtype ") + c10::toString(odtype));
        if (given) {
            on("out", *given, x, odtype);
            if (given->sizes() != at::IntArrayRef(shape) || (o[9] != Py_None && dtype_or(o[9], odtype) != odtype))
                refuse("out must be [N][H][W][C + C2] of out_dtype");
        }
        const c10::cuda::OptionalCUDAGuard guard(x.device());
        const at::Tensor out = given ? *given : new_tensor(shape, odtype, x);
        g.x = x.data_ptr();
        g.y = out.data_ptr();
        g.x_pitch = pitch_of("x", x);
        g.y_pitch = given ? pitch_of("out", out) : C;
        g.x_dtype = code_of(dtype);
        g.y_dtype = code_of(odtype);
        g.N = size32(sz[0]);
        g.H = size32(sz[1]);
        g.W = size32(sz[2]);
        g.C = size32(sz[3]);
        g.groups = as_int(o[1], "groups");
        g.act = as_int(o[5], "act");
        const double eps = PyFloat_AsDouble(o[4]);
        if (eps == -1.0 && PyErr_Occurred()) {
            PyErr_Clear();
            refuse("eps must be a number");
        }
        g.eps = (float)eps;
        return run(g_entries[o[10] == Py_True].group_norm, g, out, o[8]);
    });
}

// matmul(a, w, bias, act, residual, a2, out, out_dtype, debug)
PyObject* matmul(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 9) refuse("matmul takes 9 arguments");
        const at::Tensor &a = required(o[0], "a"), &w = required(o[1], "w");
        const at::Tensor *bias = tensor(o[2], "bias"), *residual = tensor(o[4], "residual"), *a2 = tensor(o[5], "a2"),
                         *given = tensor(o[6], "out");
        if (!a.is_cuda() || a.dim() < 1 || w.dim() != 2) refuse("a must be a CUDA tensor [...][K] and w [Nout][K + K2]");
        const at::ScalarType dtype = a.scalar_type();
        if (code_of(dtype) < 0) refuse(std::string("unsupported dtype ") + c10::toString(dtype));
        plain(&a, &w, bias, residual, a2, given);
        const auto sz = a.sizes();
        wino_matmul_args g = {};
        const int64_t K = sz[sz.size() - 1], Nout = w.size(0);
        int64_t K2 = 0;
        if (a2) {
            if (a2->dim() != a.dim() || a2->sizes().slice(0, sz.size() - 1) != sz.slice(0, sz.size() - 1))
                refuse("a2 must have a's leading dimensions");
            on("a2", *a2, a, dtype);
            K2 = a2->size(a2->dim() - 1);
            g.a2 = a2->data_ptr();
            g.a2_pitch = pitch_of("a2", *a2);
        }
        if (w.size(1) != K + K2) refuse("w has " + std::to_string(w.size(1)) + " columns, not " + std::to_string(K + K2));
        on("w", w, a, dtype);
        g.bias = param("bias", bias, a, w.sizes().slice(0, 1));
        c10::SmallVector<int64_t, 6> shape(sz.begin(), sz.end());
        shape.back() = Nout;
        const at::ScalarType odtype = given ? given->scalar_type() : dtype_or(o[7], residual ? residual->scalar_type() : dtype);
        if (code_of(odtype) < 0) refuse(std::string("unsupported output dtype ") + c10::toString(odtype));
        if (given) {
            on("out", *given, a, odtype);
            if (given->sizes() != at::IntArrayRef(shape) || (o[7] != Py_None && dtype_or(o[7], odtype) != odtype))
                refuse("out must be [...][Nout] of out_dtype");
        }
        if (residual) {
            on("residual", *residual, a, odtype);
            if (residual->sizes() != at::IntArrayRef(shape)) refuse("residual must be [...][Nout]");
            g.residual = residual->data_ptr();
            g.residual_pitch = pitch_of("residual", *residual);
        }
        const c10::cuda::OptionalCUDAGuard guard(a.device());
        const at::Tensor out = given ? *given : new_tensor(shape, odtype, a);
        g.a = a.data_ptr();
        g.w = w.data_ptr();
        g.out = out.data_ptr();
        g.a_pitch = pitch_of("a", a);
        g.w_pitch = pitch_of("w", w);
        g.out_pitch = given ? pitch_of("out", out) : Nout;
        g.dtype = code_of(dtype);
        g.out_dtype = code_of(odtype);
        g.M = K ? size32(a.numel() / K) : 0;
        g.N = size32(Nout);
        g.K = size32(K);
        g.K2 = size32(K2);
        g.act = as_int(o[3], "act");
        return run(g_entries[o[8] == Py_True].matmul, g, out, o[6]);
    });
}

// set_entries(debug, address of wino_group_norm, address of wino_matmul)
PyObject* set_entries(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (n != 3) {
        PyErr_SetString(PyExc_ValueError, "set_entries takes 3 arguments");
        return nullptr;
    }
    Entries& e = g_entries[o[0] == Py_True];
    e.group_norm = reinterpret_cast<Status>(PyLong_AsVoidPtr(o[1]));
    e.matmul = reinterpret_cast<Status>(PyLong_AsVoidPtr(o[2]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

// pitch(tensor): as the functions above take it
PyObject* pitch(PyObject*, PyObject* const* o, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (n != 1) refuse("pitch takes 1 argument");
        return PyLong_FromLongLong(pitch_of("tensor", required(o[0], "tensor")));
    });
}

PyMethodDef kMethods[] = {
    {"group_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(group_norm)), METH_FASTCALL, nullptr},
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(matmul)), METH_FASTCALL, nullptr},
    {"set_entries", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(set_entries)), METH_FASTCALL, nullptr},
    {"pitch", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(pitch)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "torch_ops_b200", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_torch_ops_b200() { return PyModule_Create(&kModule); }
