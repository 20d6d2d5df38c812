// qmm_torch.cpp -- the calls of q4g.py and q8c.py that a decode step makes many times, as
// a CPython extension: argument checks on torch tensors, output and workspace
// allocation and the library call.  (The same in Python over ctypes costs 8 to
// 18 us a call, more than the kernels; this costs about 4.)  It computes
// nothing: every kernel is libqmm.so's, through include/qmm.h.
//
// A call returns its tensor(s), or the library's status as an int when that is
// not QMM_OK (the module raises it); tensors that do not fit raise ValueError.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
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

// (up, its data, down, its data, router, x, bias, top_k, score, groups, top_groups, group_score, renorm, scale, route, out, workspace)
// -> y or (y, ids, weights)
PyObject* layer(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 17, "layer takes 17 arguments");
        int64_t device, device2;
        const qmm_q4g up = weights(a[0], a[1], device), down = weights(a[2], a[3], device2);
        need(device == device2, "both weights are on one device");
        const at::Tensor &router = tensor(a[4], "router is a tensor"), &x = tensor(a[5], "x is a tensor");
        qmm_float rt, xt;
        need(router.is_cuda() && router.get_device() == device && router.dim() == 2 && router.size(0) == up.experts && router.size(1) == up.K &&
                 router.is_contiguous() && float_type(router.scalar_type(), rt),
             "router is contiguous f32, f16 or bf16 [experts, K] on the weights' device");
        int64_t ld;
        activations(up, device, x, 2, xt, ld);
        const float* bias = nullptr;
        if (a[6] != Py_None) {
            const at::Tensor& b = tensor(a[6], "bias is a tensor");
            need(b.is_cuda() && b.get_device() == device && b.scalar_type() == at::kFloat && b.dim() == 1 && b.size(0) == up.experts && b.is_contiguous(),
                 "bias is f32 [experts] on the weights' device");
            bias = b.data_ptr<float>();
        }
        qmm_route_config cfg;
        cfg.top_k = integer32(a[7]);
        cfg.score = integer32(a[8]);
        cfg.groups = integer32(a[9]);
        cfg.top_groups = integer32(a[10]);
        cfg.group_score = integer32(a[11]);
        cfg.renorm = truth(a[12]);
        cfg.scale = (float)PyFloat_AsDouble(a[13]);
        if (PyErr_Occurred()) throw python_error();
        const bool route = truth(a[14]);
        const int64_t T = x.size(0);
        if (T > QMM_MOE_LAYER_MAX_TOKENS || cfg.top_k < 1 || cfg.top_k > QMM_MOE_MAX_TOP_K) return PyLong_FromLong(QMM_ERR_SHAPE);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        const at::Tensor y = output(a[15], {T, down.N}, x);
        at::Tensor ids, wt;
        if (route) {
            ids = empty({T, cfg.top_k}, at::kInt, x.device());
            wt = empty({T, cfg.top_k}, at::kFloat, x.device());
        }
        const Workspace ws(a[16], a[16] == Py_None ? qmm_moe_layer_workspace(&up, &down, xt, T, cfg.top_k) : 0, x);
        const qmm_status s = qmm_moe_layer(&up, &down, &cfg, rt, router.data_ptr(), bias, xt, x.data_ptr(), ld, T, y.data_ptr(),
                                           route ? ids.data_ptr<int32_t>() : nullptr, route ? wt.data_ptr<float>() : nullptr, ws.p, ws.n, stream_of(device));
        if (s != QMM_OK || !route) return result(s, y);
        PyObject* t = PyTuple_New(3);
        if (!t) return nullptr;
        PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(y));
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(ids));
        PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(wt));
        return t;
    });
}

// elements from a row of [rows, K] to the next; rows are contiguous and apart
int64_t row_distance(const at::Tensor& t, const char* text) {
    need(t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1), text);
    const int64_t ld = t.size(0) > 1 ? t.stride(0) : t.size(1);
    need(ld >= t.size(1), text);
    return ld;
}
bool on(const at::Tensor& t, int64_t device) { return t.is_cuda() && t.get_device() == device; }

at::ScalarType scalar_type(PyObject* o) {
    need(THPDtype_Check(o), "dtype is a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// (weights, their data, x, scales of the rows, bias, dtype, out, workspace)
PyObject* matmul8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 8, "matmul8 takes 8 arguments");
        qmm_q8c w = *reinterpret_cast<const qmm_q8c*>(integer(a[0]));
        const at::Tensor& data = tensor(a[1], "laid-out weights are a tensor");
        need(data.is_cuda() && data.is_contiguous() && data.nbytes() >= qmm_q8c_bytes(w.N, w.K), "the weights are on a CUDA device, whole");
        w.data = data.data_ptr();
        const int64_t device = data.get_device();
        const at::Tensor& x = tensor(a[2], "x is a tensor, or Rows8");
        const bool codes = a[3] != Py_None;
        qmm_float xt = QMM_FLOAT_F32, yt;
        const char* text = codes ? "x's codes are int8 [rows, K], rows contiguous, on the weights' device" : "activations are f32, f16 or bf16 [rows, K] on the weights' device, rows contiguous";
        need(on(x, device) && x.dim() == 2 && x.size(1) == w.K && (codes ? x.scalar_type() == at::kChar : float_type(x.scalar_type(), xt)), text);
        const int64_t M = x.size(0), ld = row_distance(x, text);
        const float* scales = nullptr;
        if (codes) {
            const at::Tensor& s = tensor(a[3], "scales are a tensor");
            need(on(s, device) && s.scalar_type() == at::kFloat && s.dim() == 1 && s.size(0) == M && s.is_contiguous(), "x's scales are f32 [rows] on the weights' device");
            scales = s.data_ptr<float>();
        }
        const float* bias = nullptr;
        if (a[4] != Py_None) {
            const at::Tensor& b = tensor(a[4], "bias is a tensor");
            need(on(b, device) && b.scalar_type() == at::kFloat && b.dim() == 1 && b.size(0) == w.N && b.is_contiguous(), "bias is f32 [N] on the weights' device");
            bias = b.data_ptr<float>();
        }
        at::ScalarType ys = a[5] != Py_None ? scalar_type(a[5]) : a[6] != Py_None ? tensor(a[6], "out is a tensor").scalar_type() : codes ? at::kFloat : x.scalar_type();
        need(float_type(ys, yt), "the result is f32, f16 or bf16");
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        at::Tensor y;
        if (a[6] == Py_None) {
            y = empty({M, w.N}, ys, x.device());
        } else {
            y = tensor(a[6], "out is a tensor");
            need(y.dim() == 2 && y.size(0) == M && y.size(1) == w.N && y.scalar_type() == ys && y.is_contiguous() && on(y, device),
                 "out is contiguous, of the result's shape, type and device");
        }
        // few values in aligned rows need no workspace (include/qmm.h)
        const bool direct = M <= QMM_Q8C_DIRECT_ROWS && w.K % 16 == 0 && w.K <= 32768 && (reinterpret_cast<uintptr_t>(x.data_ptr()) | (uintptr_t)(ld * x.element_size())) % 16 == 0 &&
                            (codes || M * w.K <= QMM_Q8C_DIRECT);
        const Workspace ws(a[7], a[7] == Py_None && !direct ? qmm_q8c_matmul_workspace(&w, codes, M) : 0, x);
        return result(qmm_q8c_matmul(&w, xt, x.data_ptr(), ld, scales, M, bias, yt, y.data_ptr(), ws.p, ws.n, stream_of(device)), y);
    });
}

// (y, weight, residual, post weight, gate, scale, eps, weight offset, quantize, out, residual out) -> (r', h) or (r', codes, scales)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        need(n == 11, "norm takes 11 arguments");
        const at::Tensor& y = tensor(a[0], "y is a tensor");
        qmm_norm p = {};
        need(y.is_cuda() && y.dim() == 2 && float_type(y.scalar_type(), p.type), "y is CUDA f32, f16 or bf16 [T, K]");
        const int64_t T = y.size(0), K = y.size(1), device = y.get_device();
        const char* text = "y, residual and outputs are [T, K] of one type and device, rows contiguous";
        auto rows = [&](const at::Tensor& t, int64_t& ld) {
            need(on(t, device) && t.sizes() == y.sizes() && t.scalar_type() == y.scalar_type(), text);
            ld = row_distance(t, text);
            return t.data_ptr();
        };
        p.y = rows(y, p.ldy);
        const at::Tensor& w = tensor(a[1], "weight is a tensor");
        need(float_type(w.scalar_type(), p.weight_type) && on(w, device) && w.dim() == 1 && w.size(0) == K && w.is_contiguous(), "weight is f32, f16 or bf16 [K] on y's device");
        p.weight = w.data_ptr();
        if (a[2] != Py_None) p.residual = rows(tensor(a[2], "residual is a tensor"), p.ldr);
        if (a[3] != Py_None) {
            const at::Tensor& t = tensor(a[3], "post_weight is a tensor");
            need(t.scalar_type() == w.scalar_type() && on(t, device) && t.sizes() == w.sizes() && t.is_contiguous(), "post_weight is as weight");
            p.post_weight = t.data_ptr();
        }
        if (a[4] != Py_None) {
            const at::Tensor& t = tensor(a[4], "gate is a tensor");
            if (t.dim() == 1) {
                need(on(t, device) && t.size(0) == K && t.scalar_type() == y.scalar_type() && t.is_contiguous(), "gate is [K] or [T, K] of y's type and device");
                p.gate = t.data_ptr();
            } else {
                p.gate = rows(t, p.ldg);
            }
        }
        p.scale = (float)PyFloat_AsDouble(a[5]);
        p.eps = (float)PyFloat_AsDouble(a[6]);
        p.weight_offset = (float)PyFloat_AsDouble(a[7]);
        if (PyErr_Occurred()) throw python_error();
        const bool quantize = truth(a[8]);
        need(!quantize || a[9] == Py_None, "quantized rows are allocated by the call: no out");
        if (K < 1 || K > QMM_NORM_MAX_K) return PyLong_FromLong(QMM_ERR_SHAPE);
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
        // Small float results share an allocation, in 16-byte steps: half of a small call's time is the memory's.
        // Results of several types have one each: torch.save takes no storage that is seen as two types.
        const at::ScalarType type = y.scalar_type();
        auto r16 = [](int64_t n) { return (n + 15) / 16 * 16; };
        const int64_t pitch = r16(K), values = r16(T * K * (int64_t)y.element_size());
        const bool both = !quantize && a[10] == Py_None && a[9] == Py_None && 2 * values <= 262144;
        at::Tensor buffer, r, h, scales;
        if (both) buffer = empty({2 * values / (int64_t)y.element_size()}, type, y.device());
        r = both ? part(buffer, 0, {T, K}) : a[10] == Py_None ? empty({T, K}, type, y.device()) : tensor(a[10], "residual_out is a tensor");
        p.residual_out = rows(r, p.ldro);
        if (quantize) {
            h = empty({T, pitch}, at::kChar, y.device());
            if (pitch != K) h.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef({T, K}), at::IntArrayRef({pitch, 1}));
            scales = empty({T}, at::kFloat, y.device());
            p.codes = static_cast<int8_t*>(h.data_ptr());
            p.scales = static_cast<float*>(scales.data_ptr());
            p.ldh = pitch;
        } else {
            h = both ? part(buffer, values / (int64_t)y.element_size(), {T, K}) : a[9] == Py_None ? empty({T, K}, type, y.device()) : tensor(a[9], "out is a tensor");
            p.h = rows(h, p.ldh);
        }
        const qmm_status s = qmm_block_norm(&p, T, K, stream_of(device));
        if (s != QMM_OK) return PyLong_FromLong(s);
        PyObject* t = PyTuple_New(quantize ? 3 : 2);
        if (!t) return nullptr;
        PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(r));
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(h));
        if (quantize) PyTuple_SET_ITEM(t, 2, THPVariable_Wrap(scales));
        return t;
    });
}

PyMethodDef methods[] = {
    {"matmul", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul)), METH_FASTCALL, nullptr},
    {"route", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(route)), METH_FASTCALL, nullptr},
    {"gate_up", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(experts<false>)), METH_FASTCALL, nullptr},
    {"down", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(experts<true>)), METH_FASTCALL, nullptr},
    {"layer", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(layer)), METH_FASTCALL, nullptr},
    {"matmul8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(matmul8)), METH_FASTCALL, nullptr},
    {"norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qmm_torch(void) { return PyModule_Create(&module); }
