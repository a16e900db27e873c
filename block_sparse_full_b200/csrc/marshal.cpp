// Argument marshalling of the paged cache and window attention for Python: checks
// the tensors, allocates outputs and workspace with torch, makes the device of
// the tensors current and calls the C entry points (ssa.h) on torch's current
// stream.  It computes nothing.  The same steps in Python took 15 to 25 us a
// call, several times the kernels of a decode step; here they take about 4.
//
// Every function takes the params structure as a buffer, tensors or None, and
// returns its outputs, or the status of the C call as an int if that failed.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "ssa.h"

namespace {

using at::Tensor;

std::string format(const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return buf;
}

// Python's ValueError and TypeError
struct ValueError : torch::PyTorchError {
    template <typename... A>
    explicit ValueError(const char* fmt, A... a) : torch::PyTorchError(format(fmt, a...)) {}
    PyObject* python_type() override { return PyExc_ValueError; }
};
struct TypeError : torch::PyTorchError {
    template <typename... A>
    explicit TypeError(const char* fmt, A... a) : torch::PyTorchError(format(fmt, a...)) {}
    PyObject* python_type() override { return PyExc_TypeError; }
};

std::string dims(c10::IntArrayRef s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + ")";
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeError("%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

template <typename P>
struct Params {  // a ctypes structure, by the buffer protocol
    Py_buffer buf{};
    explicit Params(PyObject* o) {
        if (PyObject_GetBuffer(o, &buf, PyBUF_SIMPLE) != 0) throw python_error();
        if (buf.len != (Py_ssize_t)sizeof(P)) {
            PyBuffer_Release(&buf);
            throw TypeError("params is not the structure that this call takes");
        }
    }
    ~Params() { PyBuffer_Release(&buf); }
    Params(const Params&) = delete;
    const P* operator->() const { return static_cast<const P*>(buf.buf); }
    const P* get() const { return static_cast<const P*>(buf.buf); }
};

at::ScalarType type_of(int dtype) {
    if (dtype == SSA_BF16) return at::kBFloat16;
    if (dtype == SSA_F32) return at::kFloat;
    throw ValueError("unknown dtype %d", dtype);
}

c10::Device cuda_device(const Tensor& t, const char* name) {
    if (!t.is_cuda()) throw ValueError("%s must be a CUDA tensor", name);
    return t.device();
}

void need(const Tensor& t, const char* name, c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    if (t.sizes() != shape)
        throw ValueError("%s must have shape %s, got %s", name, dims(shape).c_str(), dims(t.sizes()).c_str());
    if (t.scalar_type() != type || t.device() != dev)
        throw ValueError("%s must be %s on %s, got %s on %s", name, c10::toString(type), dev.str().c_str(),
                         c10::toString(t.scalar_type()), t.device().str().c_str());
}

// [B,H,T,D], [B,H,D] or [T,H,D] with the last axis contiguous
ssa_view_t view(const Tensor& t, const char* name, c10::IntArrayRef shape, at::ScalarType type, c10::Device dev,
                bool tokens_first = false) {
    need(t, name, shape, type, dev);
    const auto st = t.strides();
    if (st.back() != 1) throw ValueError("%s: the last axis must be contiguous (stride %lld)", name, (long long)st.back());
    if (shape.size() == 4) return {t.data_ptr(), st[0], st[1], st[2]};
    if (tokens_first) return {t.data_ptr(), 0, st[1], st[0]};
    return {t.data_ptr(), st[0], st[1], 0};
}

void* array(const Tensor& t, const char* name, c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    need(t, name, shape, type, dev);
    if (!t.is_contiguous()) throw ValueError("%s must be contiguous", name);
    return t.data_ptr();
}
void* array(PyObject* o, const char* name, c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    return array(tensor(o, name), name, shape, type, dev);
}
void* opt_array(PyObject* o, const char* name, c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    return o == Py_None ? nullptr : array(o, name, shape, type, dev);
}

void* pages(PyObject* o, const char* name, const ssa_cache_params_t* p, c10::Device dev) {
    const Tensor& t = tensor(o, name);
    need(t, name, {p->n_pages, p->Hkv, p->page, p->D}, type_of(p->dtype), dev);
    const auto st = t.strides();
    if (st[3] != 1 || st[2] != p->D || (p->Hkv > 1 && st[1] != (int64_t)p->page * p->D) ||
        (p->n_pages > 1 && st[0] != p->page_stride))
        throw ValueError("%s: each page must be contiguous and %lld elements after the one before", name,
                         (long long)p->page_stride);
    return t.data_ptr();
}

Tensor empty(c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}

struct Scratch {
    Tensor own;
    void* ptr;
    size_t bytes;
    Scratch(PyObject* o, size_t need_bytes, c10::Device dev) {
        const Tensor* t = &own;
        if (o == Py_None) {
            if (need_bytes == (size_t)-1) need_bytes = 0;  // the call itself says what is wrong
            own = empty({(int64_t)(need_bytes ? need_bytes : 1)}, at::kByte, dev);
        } else {
            t = &tensor(o, "ws");
            if (t->device() != dev || !t->is_contiguous()) throw ValueError("ws must be a contiguous tensor on %s", dev.str().c_str());
        }
        ptr = t->data_ptr();
        bytes = t->nbytes();
    }
};

// call(stream) with the tensors' device current
template <typename F>
int launch(c10::Device dev, F&& call) {
    const c10::cuda::CUDAGuard guard(dev);
    void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call(stream);
    Py_END_ALLOW_THREADS
    return status;
}

PyObject* given_or(PyObject* o, const Tensor& t) { return o == Py_None ? THPVariable_Wrap(t) : Py_NewRef(o); }
PyObject* pair(PyObject* a, PyObject* b) {
    PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

void count(Py_ssize_t n, Py_ssize_t want, const char* name) {
    if (n != want) throw TypeError("%s takes %d arguments", name, (int)want);
}

// (params, q, k, v, lens, h, lse) -> (h, lse)
PyObject* window_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7, "window_fwd");
    const Params<ssa_window_params_t> p(a[0]);
    const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    const c10::Device dev = cuda_device(q, "q");
    const auto ty = type_of(p->dtype);
    const std::initializer_list<int64_t> qs = {p->B, p->Hq, p->T, p->D}, ks = {p->B, p->Hkv, p->T, p->D}, ls = {p->B, p->Hq, p->T};
    const ssa_view_t vq = view(q, "q", qs, ty, dev), vk = view(k, "k", ks, ty, dev), vv = view(v, "v", ks, ty, dev);
    const auto* lens = static_cast<const int32_t*>(opt_array(a[4], "lens", {p->B}, at::kInt, dev));
    const Tensor h = a[5] == Py_None ? at::empty_like(q) : tensor(a[5], "h");
    const Tensor lse = a[6] == Py_None ? empty(ls, at::kFloat, dev) : tensor(a[6], "lse");
    const ssa_view_t vh = view(h, "h", qs, ty, dev);
    auto* pl = static_cast<float*>(array(lse, "lse", ls, at::kFloat, dev));
    const int st = launch(dev, [&](void* s) { return ssa_window_fwd(p.get(), &vq, &vk, &vv, lens, &vh, pl, s); });
    if (st != SSA_OK) return PyLong_FromLong(st);
    return pair(given_or(a[5], h), given_or(a[6], lse));
    END_HANDLE_TH_ERRORS
}

// (params, q, k, v, lens, h, lse, dh, ws, dq, dk, dv) -> (dq, dk, dv)
PyObject* window_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 12, "window_bwd");
    const Params<ssa_window_params_t> p(a[0]);
    const Tensor &q = tensor(a[1], "q"), &k = tensor(a[2], "k"), &v = tensor(a[3], "v");
    const c10::Device dev = cuda_device(q, "q");
    const auto ty = type_of(p->dtype);
    const std::initializer_list<int64_t> qs = {p->B, p->Hq, p->T, p->D}, ks = {p->B, p->Hkv, p->T, p->D};
    const ssa_view_t vq = view(q, "q", qs, ty, dev), vk = view(k, "k", ks, ty, dev), vv = view(v, "v", ks, ty, dev);
    const auto* lens = static_cast<const int32_t*>(opt_array(a[4], "lens", {p->B}, at::kInt, dev));
    const ssa_view_t vh = view(tensor(a[5], "h"), "h", qs, ty, dev);
    const auto* lse = static_cast<const float*>(array(a[6], "lse", {p->B, p->Hq, p->T}, at::kFloat, dev));
    const ssa_view_t vdh = view(tensor(a[7], "dh"), "dh", qs, ty, dev);
    const Scratch ws(a[8], a[8] == Py_None ? ssa_window_workspace_size(p.get()) : 0, dev);
    const Tensor dq = a[9] == Py_None ? at::empty_like(q) : tensor(a[9], "dq");
    const Tensor dk = a[10] == Py_None ? at::empty_like(k) : tensor(a[10], "dk");
    const Tensor dv = a[11] == Py_None ? at::empty_like(v) : tensor(a[11], "dv");
    const ssa_view_t vdq = view(dq, "dq", qs, ty, dev), vdk = view(dk, "dk", ks, ty, dev), vdv = view(dv, "dv", ks, ty, dev);
    const int st = launch(dev, [&](void* s) {
        return ssa_window_bwd(p.get(), &vq, &vk, &vv, lens, &vh, lse, &vdh, &vdq, &vdk, &vdv, ws.ptr, ws.bytes, s);
    });
    if (st != SSA_OK) return PyLong_FromLong(st);
    PyObject *x = given_or(a[9], dq), *y = given_or(a[10], dk), *z = given_or(a[11], dv);
    PyObject* r = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
    Py_XDECREF(x);
    Py_XDECREF(y);
    Py_XDECREF(z);
    return r;
    END_HANDLE_TH_ERRORS
}

// (params, k_pages, v_pages, table, lens, k, v, q, inv_freq, interleaved, q_start, pos_offset, new_lens, q_out, k_out)
// -> (q_out, new_lens)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 15, "cache_append");
    const Params<ssa_cache_params_t> p(a[0]);
    const Tensor &k = tensor(a[5], "k"), &v = tensor(a[6], "v");
    const c10::Device dev = cuda_device(k, "k");
    const auto ty = type_of(p->dtype);
    if (k.dim() != 3) throw ValueError("k must have shape (tokens, heads, D), got %s", dims(k.sizes()).c_str());
    const int64_t N = k.size(0);
    if (N > 0x7fffffff) throw ValueError("too many tokens");
    const std::initializer_list<int64_t> ks = {N, p->Hkv, p->D}, qs = {N, p->Hq, p->D};
    const ssa_view_t vk = view(k, "k", ks, ty, dev, true), vv = view(v, "v", ks, ty, dev, true);
    const bool has_q = a[7] != Py_None;
    if (!has_q && a[13] != Py_None) throw ValueError("q_out without q");
    ssa_view_t vq{}, vqo{}, vko{};
    Tensor q_out;
    if (has_q) {
        const Tensor& q = tensor(a[7], "q");
        vq = view(q, "q", qs, ty, dev, true);
        q_out = a[13] == Py_None ? at::empty_like(q) : tensor(a[13], "q_out");
        vqo = view(q_out, "q_out", qs, ty, dev, true);
    }
    const bool has_ko = a[14] != Py_None;
    if (has_ko) vko = view(tensor(a[14], "k_out"), "k_out", ks, ty, dev, true);
    void *kp = pages(a[1], "k_pages", p.get(), dev), *vp = pages(a[2], "v_pages", p.get(), dev);
    const auto* table = static_cast<const int32_t*>(array(a[3], "table", {p->B, p->max_pages}, at::kInt, dev));
    const auto* lens = static_cast<const int32_t*>(array(a[4], "lens", {p->B}, at::kInt, dev));
    const Tensor nl = a[12] == Py_None ? at::empty_like(tensor(a[4], "lens")) : tensor(a[12], "new_lens");
    auto* new_lens = static_cast<int32_t*>(array(nl, "new_lens", {p->B}, at::kInt, dev));
    const auto* start = static_cast<const int32_t*>(opt_array(a[10], "q_start", {(int64_t)p->B + 1}, at::kInt, dev));
    const double* freq = nullptr;
    int64_t rot = 0;
    if (a[8] != Py_None) {
        const Tensor& f = tensor(a[8], "inv_freq");
        rot = 2 * f.numel();
        if (rot > p->D) throw ValueError("inv_freq has more than D / 2 = %d values", p->D / 2);
        freq = static_cast<const double*>(array(f, "inv_freq", {f.numel()}, at::kDouble, dev));
    }
    const int inter = PyObject_IsTrue(a[9]);
    const long offset = PyLong_AsLong(a[11]);
    if (inter < 0 || (offset == -1 && PyErr_Occurred())) return nullptr;
    if (offset < 0 || offset > 0x7fffffff) throw ValueError("pos_offset must be in [0, 2^31), got %ld", offset);
    const int st = launch(dev, [&](void* s) {
        return ssa_cache_append(p.get(), (int)N, &vk, &vv, has_q ? &vq : nullptr, kp, vp, table, lens, new_lens, start,
                                freq, (int)rot, inter, (int)offset, has_q ? &vqo : nullptr, has_ko ? &vko : nullptr, s);
    });
    if (st != SSA_OK) return PyLong_FromLong(st);
    return pair(has_q ? given_or(a[13], q_out) : Py_NewRef(Py_None), given_or(a[12], nl));
    END_HANDLE_TH_ERRORS
}

// (params, q, k_pages, v_pages, prefix_pages, prefix_len, table, lens, ws, h, lse) -> (h, lse);
// prefix_pages None and prefix_len -1: ssa_paged_decode
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 11, "decode");
    const Params<ssa_cache_params_t> p(a[0]);
    const Tensor& q = tensor(a[1], "q");
    const c10::Device dev = cuda_device(q, "q");
    const auto ty = type_of(p->dtype);
    const std::initializer_list<int64_t> hs = {p->B, p->Hq, p->D}, ls = {p->B, p->Hq};
    const ssa_view_t vq = view(q, "q", hs, ty, dev);
    void *kp = pages(a[2], "k_pages", p.get(), dev), *vp = pages(a[3], "v_pages", p.get(), dev);
    const long P = PyLong_AsLong(a[5]);
    if (P == -1 && PyErr_Occurred()) return nullptr;
    if (P < -1 || P > 0x7fffffff) throw ValueError("prefix_len must be in [0, 2^31), got %ld", P);
    const int32_t* pre = nullptr;
    if (P > 0 && p->page > 0)
        pre = static_cast<const int32_t*>(array(a[4], "prefix_pages", {(P + p->page - 1) / p->page}, at::kInt, dev));
    const auto* table = static_cast<const int32_t*>(array(a[6], "table", {p->B, p->max_pages}, at::kInt, dev));
    const auto* lens = static_cast<const int32_t*>(array(a[7], "lens", {p->B}, at::kInt, dev));
    const Scratch ws(a[8], a[8] == Py_None ? ssa_cache_workspace_size(p.get(), P > 0 ? (int)P : 0) : 0, dev);
    const Tensor h = a[9] == Py_None ? at::empty_like(q) : tensor(a[9], "h");
    const Tensor lse = a[10] == Py_None ? empty(ls, at::kFloat, dev) : tensor(a[10], "lse");
    const ssa_view_t vh = view(h, "h", hs, ty, dev);
    auto* pl = static_cast<float*>(array(lse, "lse", ls, at::kFloat, dev));
    const int st = launch(dev, [&](void* s) {
        return P < 0 ? ssa_paged_decode(p.get(), &vq, kp, vp, table, lens, &vh, pl, ws.ptr, ws.bytes, s)
                     : ssa_prefix_decode(p.get(), &vq, kp, vp, pre, (int)P, table, lens, &vh, pl, ws.ptr, ws.bytes, s);
    });
    if (st != SSA_OK) return PyLong_FromLong(st);
    return pair(given_or(a[9], h), given_or(a[10], lse));
    END_HANDLE_TH_ERRORS
}

// The structure for these tensors, an instance of the ctypes class cls.
template <typename P>
PyObject* instance(PyObject* cls, const P& p) {
    PyObject* bytes = PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&p), sizeof p);
    PyObject* r = bytes ? PyObject_CallMethod(cls, "from_buffer_copy", "O", bytes) : nullptr;
    Py_XDECREF(bytes);
    return r;
}

int number(PyObject* o, const char* name) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    if (v < INT_MIN || v > INT_MAX) throw ValueError("%s does not fit into an int (%ld)", name, v);
    return (int)v;
}
float scale_of(PyObject* o, int64_t D) {
    if (o == Py_None) return (float)(1.0 / std::sqrt((double)D));
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return (float)v;
}
int dtype_of(const Tensor& t, const char* name) {
    if (t.scalar_type() == at::kBFloat16) return SSA_BF16;
    if (t.scalar_type() == at::kFloat) return SSA_F32;
    throw ValueError("%s must be bfloat16 or float32, got %s", name, c10::toString(t.scalar_type()));
}
const Tensor& ranked(PyObject* o, const char* name, int64_t dim) {
    const Tensor& t = tensor(o, name);
    if (t.dim() != dim) throw ValueError("%s must have %d axes, got shape %s", name, (int)dim, dims(t.sizes()).c_str());
    for (const int64_t n : t.sizes())
        if (n > INT_MAX) throw ValueError("%s: an axis of %lld is too long", name, (long long)n);
    return t;
}

// (cls, q, k, window, sinks, sm_scale, flags)
PyObject* window_params_for(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7, "window_params_for");
    const Tensor &q = ranked(a[1], "q", 4), &k = ranked(a[2], "k", 4);
    ssa_window_params_t p{};
    p.B = (int)q.size(0), p.Hq = (int)q.size(1), p.Hkv = (int)k.size(1), p.T = (int)q.size(2), p.D = (int)q.size(3);
    p.window = number(a[3], "window"), p.sinks = number(a[4], "sinks");
    p.dtype = dtype_of(q, "q"), p.sm_scale = scale_of(a[5], p.D), p.flags = (unsigned)number(a[6], "flags");
    return instance(a[0], p);
    END_HANDLE_TH_ERRORS
}

// (cls, q, k_pages, table, window, sinks, sm_scale)
PyObject* cache_params_for(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 7, "cache_params_for");
    const Tensor &q = tensor(a[1], "q"), &kp = ranked(a[2], "k_pages", 4), &table = ranked(a[3], "table", 2);
    if (q.dim() < 2) throw ValueError("q must have head and row axes, got shape %s", dims(q.sizes()).c_str());
    ssa_cache_params_t p{};
    p.B = (int)table.size(0), p.Hq = (int)q.size(-2), p.Hkv = (int)kp.size(1), p.D = (int)kp.size(3);
    p.page = (int)kp.size(2), p.n_pages = (int)kp.size(0), p.max_pages = (int)table.size(1);
    p.window = number(a[4], "window"), p.sinks = number(a[5], "sinks");
    p.dtype = dtype_of(kp, "k_pages"), p.sm_scale = scale_of(a[6], p.D), p.page_stride = kp.stride(0);
    return instance(a[0], p);
    END_HANDLE_TH_ERRORS
}

using FastCall = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(FastCall f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef methods[] = {
    {"window_params_for", fast(window_params_for), METH_FASTCALL, nullptr},
    {"cache_params_for", fast(cache_params_for), METH_FASTCALL, nullptr},
    {"window_fwd", fast(window_fwd), METH_FASTCALL, nullptr},
    {"window_bwd", fast(window_bwd), METH_FASTCALL, nullptr},
    {"cache_append", fast(cache_append), METH_FASTCALL, nullptr},
    {"decode", fast(decode), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module_def); }
