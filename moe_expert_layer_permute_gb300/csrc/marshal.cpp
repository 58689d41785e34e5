// marshal.cpp - torch tensors to the C ABI's moe_tensor views, for the calls that a training step makes many
// of (binding.py): a call of ten tensors takes 0.4 us here and 5 us by Python's attributes, which at the
// smallest sizes is longer than the kernels.  Arguments only: every check is the library's.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>

#include "../../include/moe_layer.h"

namespace {

// `out` from a tensor; null for None.  A tensor that the library cannot take keeps a field that it refuses:
// no data (not on a GPU), no dtype, too many dimensions.
bool view(PyObject* o, moe_tensor* out, moe_tensor** at) {
    *at = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor or None");
        return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    *at = out;
    *out = moe_tensor{};
    const bool strided = t.layout() == at::kStrided;
    switch (t.scalar_type()) {
        case at::kBFloat16: out->dtype = MOE_DT_BF16; break;
        case at::kFloat: out->dtype = MOE_DT_F32; break;
        case at::kInt: out->dtype = MOE_DT_I32; break;
        case at::kByte:
        case at::kBool: out->dtype = MOE_DT_U8; break;
        default: out->dtype = -1;
    }
    if (!strided) out->dtype = -1;
    out->ndim = (int32_t)t.dim();
    for (int64_t i = 0; strided && i < t.dim() && i < 3; ++i) {
        out->shape[i] = t.size(i);
        out->stride[i] = t.stride(i);
    }
    out->data = strided && t.is_cuda() ? t.mutable_data_ptr() : nullptr;
    return true;
}

// One call's arguments: views of its tensors, a handle's address, a stream's (None: torch's current one).
struct Args {
    moe_tensor held[10];
    moe_tensor* t[10];
    moe_scratch* workspace;
    void* stream;
};
bool read(Args* a, PyObject* const* args, Py_ssize_t n, int tensors, Py_ssize_t want, bool workspace) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return false;
    }
    try {
        for (int i = 0; i < tensors; ++i)
            if (!view(args[i], &a->held[i], &a->t[i])) return false;
        int i = tensors;
        a->workspace = nullptr;
        if (workspace) {
            a->workspace = static_cast<moe_scratch*>(PyLong_AsVoidPtr(args[i++]));
            if (PyErr_Occurred()) return false;
        }
        a->stream = args[i] == Py_None ? (void*)c10::cuda::getCurrentCUDAStream().stream() : PyLong_AsVoidPtr(args[i]);
        return !PyErr_Occurred();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return false;
    }
}

PyObject* balance_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a;
    if (!read(&a, args, n, 7, 9, true)) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = moe_balance_fwd(a.t[0], a.t[1], a.t[2], a.t[3], a.t[4], a.t[5], a.t[6], a.workspace, a.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

PyObject* balance_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a;
    if (!read(&a, args, n, 10, 11, false)) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = moe_balance_bwd(a.t[0], a.t[1], a.t[2], a.t[3], a.t[4], a.t[5], a.t[6], a.t[7], a.t[8], a.t[9], a.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// G, O, workspace, stream, steps, eps, and 3 * steps coefficients (or none)
PyObject* orthogonalise(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a;
    if (n < 6) {
        PyErr_SetString(PyExc_TypeError, "expected six arguments and the coefficients");
        return nullptr;
    }
    const long steps = PyLong_AsLong(args[4]);
    if (PyErr_Occurred()) return nullptr;
    const double eps = PyFloat_AsDouble(args[5]);
    if (PyErr_Occurred()) return nullptr;
    float co[3 * MOE_ORTHOGONALISE_MAX_STEPS];
    const Py_ssize_t given = n - 6;
    if (given != 0 && (steps < 1 || given != 3 * steps || steps > MOE_ORTHOGONALISE_MAX_STEPS))
        return PyLong_FromLong(steps < 1 || given != 3 * steps ? MOE_ERR_SHAPE : MOE_ERR_UNSUPPORTED);
    for (Py_ssize_t i = 0; i < given; ++i) co[i] = (float)PyFloat_AsDouble(args[6 + i]);   // given <= the array's size
    if (PyErr_Occurred() || !read(&a, args, 4, 2, 4, true)) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = moe_orthogonalise(a.t[0], a.t[1], (int32_t)std::clamp<long>(steps, INT32_MIN, INT32_MAX), given ? co : nullptr, (float)eps,
                           a.workspace, a.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// The arguments of calls that may be on any device: tensors of one of them, whose current stream is taken where none is
// given, and which is the current device during the call.  `at` is where the stream stands.
struct On {
    c10::cuda::OptionalCUDAGuard guard;
    void* stream = nullptr;
};
bool read_on(Args* a, On* on, PyObject* const* args, Py_ssize_t n, int tensors, Py_ssize_t want) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return false;
    }
    try {
        int device = -1;
        for (int i = 0; i < tensors; ++i) {
            if (!view(args[i], &a->held[i], &a->t[i])) return false;
            if (args[i] == Py_None || !THPVariable_Unpack(args[i]).is_cuda()) continue;
            const int d = THPVariable_Unpack(args[i]).get_device();
            if (device >= 0 && d != device) {
                PyErr_SetString(PyExc_ValueError, "tensors of several devices");
                return false;
            }
            device = d;
        }
        if (device >= 0) on->guard.set_index((c10::DeviceIndex)device);
        PyObject* stream = args[want - 1];
        on->stream = stream == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream() : PyLong_AsVoidPtr(stream);
        return !PyErr_Occurred();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return false;
    }
}

// logits, bias, mask, topk_idx, topk_w, rule, stream
PyObject* select_fwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a;
    On on;
    if (!read_on(&a, &on, args, n, 5, 7)) return nullptr;
    const auto* rule = static_cast<const moe_router_rule*>(PyLong_AsVoidPtr(args[5]));
    if (PyErr_Occurred()) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = moe_router_select_fwd(a.t[0], a.t[1], a.t[2], a.t[3], a.t[4], rule, on.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// logits, topk_idx, topk_w, dtopk_w, dlogits, rule, accumulate, stream
PyObject* select_bwd(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a;
    On on;
    if (!read_on(&a, &on, args, n, 5, 8)) return nullptr;
    const auto* rule = static_cast<const moe_router_rule*>(PyLong_AsVoidPtr(args[5]));
    if (PyErr_Occurred()) return nullptr;
    const int accumulate = PyObject_IsTrue(args[6]);
    if (accumulate < 0) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = moe_router_select_bwd(a.t[0], a.t[1], a.t[2], a.t[3], a.t[4], rule, accumulate, on.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

// counts, bias, rate, stream
PyObject* bias_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
    Args a;
    On on;
    if (!read_on(&a, &on, args, n, 2, 4)) return nullptr;
    const double rate = PyFloat_AsDouble(args[2]);
    if (PyErr_Occurred()) return nullptr;
    int rc;
    Py_BEGIN_ALLOW_THREADS;
    rc = moe_router_bias_step(a.t[0], a.t[1], (float)rate, on.stream);
    Py_END_ALLOW_THREADS;
    return PyLong_FromLong(rc);
}

#define MOE_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"balance_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(balance_fwd)), METH_FASTCALL, nullptr},
    {"balance_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(balance_bwd)), METH_FASTCALL, nullptr},
    {"orthogonalise", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(orthogonalise)), METH_FASTCALL, nullptr},
    MOE_METHOD(select_fwd),
    MOE_METHOD(select_bwd),
    MOE_METHOD(bias_step),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
