// qmm_torch.cpp -- the calls of q4g.py that a decode step makes many times, as
// a CPython extension: argument checks on torch tensors, output and workspace
// allocation and the library call.  (The same in Python over ctypes costs 8 to
// 18 us a call, more than the kernels; this costs about 4.)  It computes
// nothing: every kernel is libqmm.so's, through include/qmm.h.
//
// A call returns its tensor(s), or the library's status as an int when that is
// not QMM_OK (q4g.py raises it); tensors that do not fit raise ValueError.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <stdexcept>

#include "../../include/qmm.h"

namespace {

struct Misfit : std::invalid_argument {
    using std::invalid_argument::invalid_argument;
};
void need(bool ok, const char* text) {
    if (!ok) throw Misfit(text);
}

bool float_type(at::ScalarType t, qmm_float& f) {
    if (t == at::kFloat) f = QMM_FLOAT_F32;
    else if (t == at::kHalf) f = QMM_FLOAT_F16;
    else if (t == at::kBFloat16) f = QMM_FLOAT_BF16;
    else return false;
    return true;
}

const at::Tensor& tensor(PyObject* o, const char* text) {
    need(THPVariable_Check(o), text);
    return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}
// an integer of the C ABI's 32 bits; what does not fit stays out of every valid range
int32_t integer32(PyObject* o) { return (int32_t)std::min<int64_t>(std::max<int64_t>(integer(o), INT32_MIN), INT32_MAX); }
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v == 1;
}
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType t, const at::Device& d) {
    return at::detail::empty_cuda(sizes, t, d, std::nullopt);
}

// `sizes` elements of a buffer from element `at` on, as a tensor of their own (a fifth of an allocation's time)
at::Tensor part(const at::Tensor& buffer, int64_t at, at::IntArrayRef sizes) {
    at::Tensor v = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buffer.storage()), buffer.key_set(), buffer.dtype());
    v.unsafeGetTensorImpl()->set_storage_offset(at);
    v.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
    return v;
}

// the weights that `o` describes, at where their tensor's data is now; the tensor's device
qmm_q4g weights(PyObject* o, PyObject* data, int64_t& device) {
    qmm_q4g w = *reinterpret_cast<const qmm_q4g*>(integer(o));
    const at::Tensor& t = tensor(data, "laid-out weights are a tensor");
    need(t.is_cuda() && t.is_contiguous() && t.nbytes() >= qmm_q4g_bytes(w.experts, w.N, w.K, w.group, w.paired),
         "the weights are on a CUDA device, whole");
    device = t.get_device();
    w.data = t.data_ptr();
    return w;
}

// type and row distance (elements) of activations [.., K]: rows contiguous and evenly apart
void activations(const qmm_q4g& w, int64_t device, const at::Tensor& x, int64_t dims, qmm_float& xt, int64_t& ld) {
    need(x.is_cuda() && x.get_device() == device && x.dim() == dims && x.size(dims - 1) == w.K && float_type(x.scalar_type(), xt),
         dims == 2 ? "activations are f32, f16 or bf16 [rows, K] on the weights' device"
                   : "activations are f32, f16 or bf16 [tokens, top_k, K] on the weights' device");
    ld = w.K;
    if (x.is_contiguous()) return;
    need(x.stride(dims - 1) == 1 && (dims == 2 || x.size(1) == 1 || x.size(0) == 1 || x.stride(0) == x.size(1) * x.stride(1)),
         "rows of activations are contiguous and evenly apart");
    ld = dims == 2 || x.size(1) == 1 ? x.stride(0) : x.stride(1);
}

at::Tensor output(PyObject* o, at::IntArrayRef sizes, const at::Tensor& x) {
    if (o == Py_None) return empty(sizes, x.scalar_type(), x.device());
    const at::Tensor& t = tensor(o, "out is a tensor");
    need(t.sizes() == sizes && t.scalar_type() == x.scalar_type() && t.is_contiguous() && t.device() == x.device(),
         "out is contiguous, of the result's shape and the activations' type and device");
    return t;
}

// a caller's workspace (the library checks its size and alignment; its bytes have to be one piece of
// this device's memory), else a new one
struct Workspace {
    at::Tensor t;
    void* p = nullptr;
    size_t n = 0;
    Workspace(PyObject* o, size_t size, const at::Tensor& like) {
        if (o != Py_None) {
            t = tensor(o, "workspace is a tensor");
            need(t.is_cuda() && t.device() == like.device() && t.is_contiguous(), "workspace is a contiguous tensor on the activations' device");
        } else if (size) {
            t = empty({(int64_t)size}, at::kByte, like.device());
        } else {
            return;
        }
        p = t.data_ptr();
        n = t.nbytes();
    }
};

qmm_stream_t stream_of(int64_t device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

PyObject* result(qmm_status s, const at::Tensor& t) { return s == QMM_OK ? THPVariable_Wrap(t) : PyLong_FromLong(s); }

// no exception leaves an entry
template <class F>
PyObject* guarded(F f) {
    HANDLE_TH_ERRORS
    try {
        return f();
    } catch (const Misfit& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// (weights, their data, x, out, workspace)
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 5, "matmul takes 5 arguments");
        int64_t device;
        const qmm_q4g w = weights(a[0], a[1], device);
        const at::Tensor& x = tensor(a[2], "x is a tensor");
        qmm_float xt;
        int64_t ld;
        activations(w, device, x, 2, xt, ld);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        const int64_t M = x.size(0);
        const at::Tensor y = output(a[3], {M, w.N}, x);
        const Workspace ws(a[4], a[4] == Py_None ? qmm_q4g_matmul_workspace(&w, xt, M) : 0, x);
        return result(qmm_q4g_matmul(&w, xt, x.data_ptr(), ld, M, y.data_ptr(), ws.p, ws.n, stream_of(device)), y);
    });
}

bool index_tensor(const at::Tensor& t, int64_t device) {
    return t.is_cuda() && t.get_device() == device && t.scalar_type() == at::kInt && t.is_contiguous();
}

// (weights, their data, x, ids, route weights, offsets, order, out, workspace)
template <bool DOWN>
PyObject* experts(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 9, "9 arguments");
        int64_t device;
        const qmm_q4g w = weights(a[0], a[1], device);
        const at::Tensor& x = tensor(a[2], "activations are a tensor");
        qmm_float xt;
        int64_t ld;
        activations(w, device, x, DOWN ? 3 : 2, xt, ld);
        const char* text = "a Route has int32 ids [T, top_k], f32 weights, int32 offsets [experts + 1] and order [T top_k], contiguous, on the weights' device";
        const at::Tensor &ids = tensor(a[3], text), &wt = tensor(a[4], text), &off = tensor(a[5], text), &order = tensor(a[6], text);
        need(index_tensor(ids, device) && index_tensor(off, device) && index_tensor(order, device) && ids.dim() == 2 &&
                 off.numel() == w.experts + 1 && order.numel() == ids.numel() && wt.is_cuda() && wt.get_device() == device &&
                 wt.scalar_type() == at::kFloat && wt.is_contiguous() && wt.sizes() == ids.sizes(),
             text);
        const int64_t T = ids.size(0), k = ids.size(1);
        need(x.size(0) == T && (!DOWN || x.size(1) == k), "route and activations have the same tokens and slots");
        const qmm_routing r = {ids.data_ptr<int32_t>(), wt.data_ptr<float>(), off.data_ptr<int32_t>(), order.data_ptr<int32_t>(), T, k};
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        if (DOWN) {
            const at::Tensor y = output(a[7], {T, w.N}, x);
            const Workspace ws(a[8], a[8] == Py_None ? qmm_moe_down_workspace(&w, xt, T, k) : 0, x);
            return result(qmm_moe_down(&w, xt, x.data_ptr(), ld, &r, y.data_ptr(), ws.p, ws.n, stream_of(device)), y);
        }
        const at::Tensor h = output(a[7], {T, k, w.N / 2}, x);
        const Workspace ws(a[8], a[8] == Py_None ? qmm_moe_gate_up_workspace(&w, xt, T, k) : 0, x);
        return result(qmm_moe_gate_up(&w, xt, x.data_ptr(), ld, &r, h.data_ptr(), ws.p, ws.n, stream_of(device)), h);
    });
}

// (logits, bias, top_k, score, groups, top_groups, group_score, renorm, scale, order, workspace) -> (ids, weights, offsets, order)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 11, "route takes 11 arguments");
        const at::Tensor& l = tensor(a[0], "logits are a tensor");
        qmm_float t;
        need(l.is_cuda() && l.dim() == 2 && float_type(l.scalar_type(), t) && (l.size(1) <= 1 || l.stride(1) == 1),
             "logits are CUDA f32, f16 or bf16 [T, experts], rows contiguous");
        const int64_t T = l.size(0), E = l.size(1), device = l.get_device(), ld = T > 1 ? l.stride(0) : E;
        const float* bias = nullptr;
        if (a[1] != Py_None) {
            const at::Tensor& b = tensor(a[1], "bias is a tensor");
            need(b.is_cuda() && b.get_device() == device && b.scalar_type() == at::kFloat && b.dim() == 1 && b.size(0) == E && b.is_contiguous(),
                 "bias is f32 [experts] on the logits' device");
            bias = b.data_ptr<float>();
        }
        qmm_route_config cfg;
        cfg.top_k = integer32(a[2]);
        cfg.score = integer32(a[3]);
        cfg.groups = integer32(a[4]);
        cfg.top_groups = integer32(a[5]);
        cfg.group_score = integer32(a[6]);
        cfg.renorm = truth(a[7]);
        cfg.scale = (float)PyFloat_AsDouble(a[8]);
        if (PyErr_Occurred()) throw python_error();
        const bool sorted = truth(a[9]);
        // what the library refuses whatever else it is given: not first the memory for it
        if (E < 1 || E > QMM_MOE_MAX_EXPERTS || cfg.top_k < 1 || cfg.top_k > QMM_MOE_MAX_TOP_K || cfg.top_k > E) return PyLong_FromLong(QMM_ERR_SHAPE);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        const int64_t k = cfg.top_k;
        // the integers are parts of one allocation, in 16-byte steps: ids, offsets, order.  The weights are not one:
        // torch.save takes no storage that is seen as two types
        const at::Tensor wt = empty({T, k}, at::kFloat, l.device());
        at::Tensor ids, off, order;
        if (sorted) {
            const int64_t n1 = (T * k + 3) / 4 * 4, n2 = (E + 4) / 4 * 4;
            const at::Tensor all = empty({2 * n1 + n2}, at::kInt, l.device());
            ids = part(all, 0, {T, k});
            off = part(all, n1, {E + 1});
            order = part(all, n1 + n2, {T * k});
        } else {
            ids = empty({T, k}, at::kInt, l.device());
        }
        const Workspace ws(a[10], sorted && a[10] == Py_None ? qmm_moe_route_workspace(T, E, k) : 0, l);
        const qmm_status s = qmm_moe_route(&cfg, t, l.data_ptr(), ld, T, E, bias, ids.data_ptr<int32_t>(), wt.data_ptr<float>(),
                                           sorted ? off.data_ptr<int32_t>() : nullptr, sorted ? order.data_ptr<int32_t>() : nullptr, ws.p,
                                           ws.n, stream_of(device));
        if (s != QMM_OK) return PyLong_FromLong(s);
        PyObject* r = PyTuple_New(4);
        if (!r) return nullptr;
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(ids));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(wt));
        PyTuple_SET_ITEM(r, 2, sorted ? THPVariable_Wrap(off) : Py_NewRef(Py_None));
        PyTuple_SET_ITEM(r, 3, sorted ? THPVariable_Wrap(order) : Py_NewRef(Py_None));
        return r;
    });
}

PyMethodDef methods[] = {
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL, nullptr},
    {"gate_up", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(experts<false>)), METH_FASTCALL, nullptr},
    {"down", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(experts<true>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_torch(void) { return PyModule_Create(&module); }
