// marshal.cpp - torch tensors to the C ABI's moe_tensor views, for the calls that a training step makes many
// of (binding.py): a call of ten tensors takes 0.4 us here and 5 us by Python's attributes, which at the
// smallest sizes is longer than the kernels.  Arguments only: every check is the library's.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <limits>
#include <memory>
#include <utility>
#include <vector>

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

// ---- lists of tensors ----
// Views of a list's tensors, made once for as many calls as there are.  The tensors are held, and each call looks whether
// they are still what the views say: a tensor may get another size, order, type or device, with or without
// another address.  Then new views are made; a call under way in another thread keeps those that it has.
struct Seen {                      // of a tensor: what its view and the list's device follow from
    const void* at;
    int64_t count;
    caffe2::TypeMeta type;
    bool contiguous;
    c10::Device device;
    explicit Seen(const c10::TensorImpl& t)
        : at(t.data()), count(t.numel()), type(t.dtype()), contiguous(t.is_contiguous()), device(t.device()) {}
    bool holds(const c10::TensorImpl& t) const {
        return t.numel() == count && t.data() == at && t.is_contiguous() == contiguous && t.dtype() == type && t.device() == device;
    }
};
using Views = std::shared_ptr<const std::vector<moe_tensor>>;
struct List {
    std::vector<at::Tensor> held;
    std::vector<std::pair<const c10::TensorImpl*, Seen>> seen;   // of the strided ones (others are refused, and stay what they are)
    Views views;
    int device = -1;               // -2: of several devices
};
// a contiguous tensor of any shape as its elements in a row
moe_tensor flat(const at::Tensor& t) {
    moe_tensor v{};
    v.ndim = 1;
    const bool strided = t.layout() == at::kStrided;
    v.shape[0] = strided ? t.numel() : 0;
    v.stride[0] = strided && t.is_contiguous() ? 1 : 2;
    switch (t.scalar_type()) {
        case at::kBFloat16: v.dtype = MOE_DT_BF16; break;
        case at::kFloat: v.dtype = MOE_DT_F32; break;
        case at::kInt: v.dtype = MOE_DT_I32; break;
        case at::kByte: v.dtype = MOE_DT_U8; break;
        case at::kFloat8_e4m3fn: v.dtype = MOE_DT_E4M3; break;
        default: v.dtype = -1;
    }
    if (!strided) v.dtype = -1;
    v.data = strided && t.is_cuda() && t.numel() ? t.mutable_data_ptr() : nullptr;
    return v;
}
void look(List* l) {
    auto views = std::make_shared<std::vector<moe_tensor>>();
    decltype(l->seen) seen;
    views->reserve(l->held.size());
    seen.reserve(l->held.size());
    int device = -1;
    for (const at::Tensor& t : l->held) {
        views->push_back(flat(t));
        if (t.layout() == at::kStrided) seen.emplace_back(t.unsafeGetTensorImpl(), Seen(*t.unsafeGetTensorImpl()));
        if (t.is_cuda()) device = device == -1 || device == t.get_device() ? (int)t.get_device() : -2;
    }
    l->seen.swap(seen);   // (all of it or nothing: whatever throws does so before)
    l->views = std::move(views);
    l->device = device;
}
constexpr char kListName[] = "moe_tensor_list";
List* list_of(PyObject* o) { return static_cast<List*>(PyCapsule_GetPointer(o, kListName)); }

PyObject* make_list(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 1) {
        PyErr_SetString(PyExc_TypeError, "expected a sequence of tensors");
        return nullptr;
    }
    PyObject* seq = PySequence_Fast(args[0], "expected a sequence of tensors");
    if (!seq) return nullptr;
    PyObject* made = nullptr;
    try {
        auto l = std::make_unique<List>();
        const Py_ssize_t count = PySequence_Fast_GET_SIZE(seq);
        l->held.reserve(count);
        for (Py_ssize_t i = 0; i < count; ++i) {
            PyObject* o = PySequence_Fast_GET_ITEM(seq, i);
            if (!THPVariable_Check(o)) {
                PyErr_SetString(PyExc_TypeError, "expected a sequence of tensors");
                Py_DECREF(seq);
                return nullptr;
            }
            l->held.push_back(THPVariable_Unpack(o));
        }
        look(l.get());
        made = PyCapsule_New(l.get(), kListName, [](PyObject* c) { delete list_of(c); });
        if (made) l.release();
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    Py_DECREF(seq);
    return made;
}

// A call's lists: of one length and one device, whose current stream is taken where none is given.
struct Lists {
    Views of[7];
    Py_ssize_t count = -1;
    int device = -1;
    bool add(int i, PyObject* o) {
        if (o == Py_None) return true;
        List* l = list_of(o);
        if (!l) return false;
        if (count < 0) count = (Py_ssize_t)l->held.size();
        if ((Py_ssize_t)l->held.size() != count) {
            PyErr_SetString(PyExc_ValueError, "lists of different lengths");
            return false;
        }
        for (const auto& [t, as] : l->seen)
            if (!as.holds(*t)) {
                look(l);
                break;
            }
        of[i] = l->views;
        return on(l->device);
    }
    bool on(int d) {
        if (d == -1) return true;
        if (d == -2 || (device >= 0 && d != device)) {
            PyErr_SetString(PyExc_ValueError, "tensors of several devices");
            return false;
        }
        device = d;
        return true;
    }
    const moe_tensor* views(int i) const { return of[i] ? of[i]->data() : nullptr; }
};
// a number on the device, or None
bool number(PyObject* o, moe_tensor* held, const moe_tensor** at, Lists* lists) {
    *at = nullptr;
    if (o == Py_None) return true;
    if (!THPVariable_Check(o)) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor or None");
        return false;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    *held = flat(t);
    *at = held;
    return !t.is_cuda() || lists->on((int)t.get_device());
}

// params, grads, m, v, m_scales, v_scales, copies (lists), lr, beta1, beta2, eps, weight_decay, step, seed, lr, step and
// grad_scale on the device, stream
PyObject* adamw_step(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 18) {
        PyErr_Format(PyExc_TypeError, "expected 18 arguments, got %zd", n);
        return nullptr;
    }
    try {
        Lists l;
        for (int i = 0; i < 7; ++i)
            if (!l.add(i, args[i])) return nullptr;
        moe_adamw_options o{};
        double* of[5] = {&o.lr, &o.beta1, &o.beta2, &o.eps, &o.weight_decay};
        for (int i = 0; i < 5; ++i) {
            *of[i] = PyFloat_AsDouble(args[7 + i]);
            if (PyErr_Occurred()) return nullptr;
        }
        o.step = PyLong_AsLongLong(args[12]);
        if (PyErr_Occurred()) return nullptr;
        o.seed = PyLong_AsUnsignedLongLongMask(args[13]);
        if (PyErr_Occurred()) return nullptr;
        moe_tensor held[3];
        if (!number(args[14], &held[0], &o.lr_on_device, &l) || !number(args[15], &held[1], &o.step_on_device, &l) ||
            !number(args[16], &held[2], &o.grad_scale, &l))
            return nullptr;
        c10::cuda::OptionalCUDAGuard guard;
        if (l.device >= 0) guard.set_index((c10::DeviceIndex)l.device);
        void* stream = args[17] == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)l.device).stream() : PyLong_AsVoidPtr(args[17]);
        if (PyErr_Occurred()) return nullptr;
        int rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = moe_adamw_step(l.count < 0 ? 0 : l.count, l.views(0), l.views(1), l.views(2), l.views(3), l.views(4), l.views(5), l.views(6), &o,
                            stream);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// grads (a list), out, max_norm, workspace, stream
PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (n != 5) {
        PyErr_Format(PyExc_TypeError, "expected 5 arguments, got %zd", n);
        return nullptr;
    }
    try {
        Lists l;
        if (!l.add(0, args[0])) return nullptr;
        moe_tensor held;
        const moe_tensor* out;
        if (!number(args[1], &held, &out, &l)) return nullptr;
        const double most = PyFloat_AsDouble(args[2]);
        if (PyErr_Occurred()) return nullptr;
        // (0 would be no clipping)
        const float max_norm = most > 0.0 && (float)most == 0.f ? std::numeric_limits<float>::denorm_min() : (float)most;
        auto* workspace = static_cast<moe_scratch*>(PyLong_AsVoidPtr(args[3]));
        if (PyErr_Occurred()) return nullptr;
        c10::cuda::OptionalCUDAGuard guard;
        if (l.device >= 0) guard.set_index((c10::DeviceIndex)l.device);
        void* stream = args[4] == Py_None ? (void*)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)l.device).stream() : PyLong_AsVoidPtr(args[4]);
        if (PyErr_Occurred()) return nullptr;
        int rc;
        Py_BEGIN_ALLOW_THREADS;
        rc = moe_grad_norm(l.count < 0 ? 0 : l.count, l.views(0), const_cast<moe_tensor*>(out), max_norm, workspace, stream);
        Py_END_ALLOW_THREADS;
        return PyLong_FromLong(rc);
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

#define MOE_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"balance_fwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(balance_fwd)), METH_FASTCALL, nullptr},
    {"balance_bwd", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(balance_bwd)), METH_FASTCALL, nullptr},
    {"orthogonalise", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(orthogonalise)), METH_FASTCALL, nullptr},
    MOE_METHOD(select_fwd),
    MOE_METHOD(select_bwd),
    MOE_METHOD(bias_step),
    MOE_METHOD(make_list),
    MOE_METHOD(adamw_step),
    MOE_METHOD(grad_norm),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
