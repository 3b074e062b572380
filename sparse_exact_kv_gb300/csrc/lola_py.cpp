// Argument marshalling of ExactAttention's calls: through Python attributes and ctypes a call costs 18 us of
// the host's time, more than the GPU's for a single token (through Python attributes in C 12-14 us).
// Each function reads what lola.h asks for from the tensors themselves, allocates the output through torch
// and makes the call on torch's current stream.  Whatever it does not take for granted -- an object that is no
// plain tensor, another shape, type or device, a refusal by the library, an exception of torch's -- makes it
// return NotImplemented with nothing enqueued: the Python form of the same call then says what is wrong, or
// handles it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>

#include "lola.h"

namespace {

using at::Tensor;

// the tensor of a Python object on `device` of type `dtype`, or null
const Tensor* get(PyObject* o, at::ScalarType dtype, int device) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda() || t.get_device() != device || t.scalar_type() != dtype) return nullptr;
    return &t;
}

// New memory of torch's, without its dispatch of operators (which takes as long as the allocation): a tensor, one like q,
// and a workspace on the current device and stream.
Tensor empty(at::IntArrayRef size, at::ScalarType dtype, int device) {
    return at::detail::empty_cuda(size, dtype, at::Device(at::kCUDA, (c10::DeviceIndex)device), std::nullopt);
}
Tensor like(const Tensor& q) { return q.is_contiguous() ? empty(q.sizes(), q.scalar_type(), q.get_device()) : at::empty_like(q); }
at::DataPtr scratch(int64_t bytes) { return c10::cuda::CUDACachingAllocator::get()->allocate((size_t)bytes); }

// a contiguous vector of n entries (n < 0: any number)
const Tensor* vec(PyObject* o, at::ScalarType dtype, int device, int64_t n) {
    const Tensor* t = get(o, dtype, device);
    return t && t->dim() == 1 && (n < 0 || t->size(0) == n) && (t->stride(0) == 1 || t->size(0) <= 1) && t->size(0) <= INT32_MAX ? t : nullptr;
}

// A layer as ExactAttention keeps it, (address of its lola_attn_config, workspace bytes), and where the call runs.
struct Call {
    const lola_attn_config* cfg;
    int64_t ws;
    int device;
    at::ScalarType dtype;
    c10::cuda::CUDAStream stream;
};
std::optional<Call> begin(PyObject* t) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 2) return std::nullopt;
    const auto* cfg = (const lola_attn_config*)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(t, 0));
    const int64_t ws = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 1));
    if (PyErr_Occurred() || !cfg || c10::cuda::device_count() == 0) return std::nullopt;
    const int device = c10::cuda::current_device();
    return Call{cfg, ws, device, cfg->dtype == LOLA_BF16 ? at::kBFloat16 : at::kFloat, c10::cuda::getCurrentCUDAStream(device)};
}

// [n, heads, d] rows (n < 0: any number)
bool fill(const Tensor& t, lola_rows* r, int64_t n, int64_t heads, int64_t d) {
    if (t.dim() != 3 || (n >= 0 && t.size(0) != n) || t.size(1) != heads || t.size(2) != d || t.stride(2) != 1 || t.size(0) > INT32_MAX)
        return false;
    r->data = t.data_ptr();
    r->head = heads == 1 ? d : t.stride(1);
    r->row = t.size(0) == 1 ? heads * r->head : t.stride(0);
    return true;
}
const Tensor* rows(PyObject* o, lola_rows* r, const Call& c, int64_t n, int64_t heads) {
    const Tensor* t = get(o, c.dtype, c.device);
    return t && fill(*t, r, n, heads, c.cfg->d) ? t : nullptr;
}

// contiguous pools [n_pages, Hkv, page, d] of one shape, and what a call has for them
bool pools(PyObject* k_pool, PyObject* v_pool, int device, const lola_attn_config* cfg, lola_paged_kv* kv, at::ScalarType type) {
    const Tensor *k = get(k_pool, type, device), *v = get(v_pool, type, device);
    if (!k || !v || k->dim() != 4 || k->size(1) != cfg->Hkv || k->size(3) != cfg->d || k->sizes() != v->sizes() || !k->is_contiguous() ||
        !v->is_contiguous() || k->size(0) > INT32_MAX || k->size(2) > INT32_MAX)
        return false;
    kv->K = k->data_ptr();
    kv->V = v->data_ptr();
    kv->n_pages = (int32_t)k->size(0);
    kv->page = (int32_t)k->size(2);
    return true;
}
// ... and a quantised cache's powers of two [n_pages, Hkv, page], contiguous
bool powers(PyObject* k_scale, PyObject* v_scale, int device, const lola_attn_config* cfg, const lola_paged_kv& kv, lola_kv_scales* sc) {
    const Tensor *k = get(k_scale, at::kFloat8_e8m0fnu, device), *v = get(v_scale, at::kFloat8_e8m0fnu, device);
    for (const Tensor* t : {k, v})
        if (!t || t->dim() != 3 || t->size(0) != kv.n_pages || t->size(1) != cfg->Hkv || t->size(2) != kv.page || !t->is_contiguous())
            return false;
    sc->K = k->data_ptr();
    sc->V = v->data_ptr();
    return true;
}
bool cache(PyObject* k_pool, PyObject* v_pool, PyObject* kv_len, PyObject* table, const Call& c, lola_paged_kv* kv,
           at::ScalarType type) {
    const Tensor* t = get(table, at::kInt, c.device);
    if (!pools(k_pool, v_pool, c.device, c.cfg, kv, type) || !t || t->dim() != 2 || (t->stride(1) != 1 && t->size(1) != 1) ||
        t->size(0) > INT32_MAX || t->size(1) > INT32_MAX)
        return false;
    const Tensor* n = vec(kv_len, at::kInt, c.device, t->size(0));
    if (!n) return false;
    kv->n_seq = (int32_t)t->size(0);
    kv->width = (int32_t)t->size(1);
    kv->table_stride = t->size(0) == 1 ? t->size(1) : t->stride(0);
    kv->table = (const int32_t*)t->data_ptr();
    kv->kv_len = (const int32_t*)n->data_ptr();
    return true;
}

bool cache(PyObject* k_pool, PyObject* v_pool, PyObject* kv_len, PyObject* table, const Call& c, lola_paged_kv* kv) {
    return cache(k_pool, v_pool, kv_len, table, c, kv, c.dtype);
}
// ... quantised
bool cache(PyObject* k_pool, PyObject* v_pool, PyObject* k_scale, PyObject* v_scale, PyObject* kv_len, PyObject* table, const Call& c,
           lola_paged_kv* kv, lola_kv_scales* sc) {
    return cache(k_pool, v_pool, kv_len, table, c, kv, at::kFloat8_e4m3fn) && powers(k_scale, v_scale, c.device, c.cfg, *kv, sc);
}

PyObject* decline() {
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

// No exception of torch's (out of memory, say) leaves a function: the Python form meets it again.
template <typename F> PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        return decline();
    }
}

// prefill(layer, q, k, v, cu_q, cu_k | None) -> out
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == 6 ? begin(a[0]) : std::nullopt;
        if (!c) return decline();
        lola_rows rq, rk, rv, ro;
        const Tensor *q = rows(a[1], &rq, *c, -1, c->cfg->Hq), *k = rows(a[2], &rk, *c, -1, c->cfg->Hkv);
        if (!q || !k || !rows(a[3], &rv, *c, k->size(0), c->cfg->Hkv)) return decline();
        const Tensor *cq = vec(a[4], at::kInt, c->device, -1), *ck = nullptr;
        if (!cq || (a[5] != Py_None && !(ck = vec(a[5], at::kInt, c->device, cq->size(0))))) return decline();
        Tensor out = like(*q);
        if (!fill(out, &ro, q->size(0), c->cfg->Hq, c->cfg->d)) return decline();
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        s = lola_attn_prefill(c->cfg, (int32_t)cq->size(0) - 1, (int32_t)q->size(0), (int32_t)k->size(0), (const int32_t*)cq->data_ptr(),
                              ck ? (const int32_t*)ck->data_ptr() : nullptr, &rq, &rk, &rv, &ro, nullptr, c->stream.stream());
        Py_END_ALLOW_THREADS
        return s == LOLA_OK ? THPVariable_Wrap(std::move(out)) : decline();
    });
}

// prefill_paged(layer, k_pool, v_pool, q, cu_q, kv_len, table, total_k) -> out
PyObject* prefill_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == 8 ? begin(a[0]) : std::nullopt;
        lola_paged_kv kv;
        if (!c || !cache(a[1], a[2], a[5], a[6], *c, &kv)) return decline();
        const long long total_k = PyLong_Check(a[7]) ? PyLong_AsLongLong(a[7]) : -1;
        lola_rows rq, ro;
        const Tensor *q = rows(a[3], &rq, *c, -1, c->cfg->Hq), *cq = vec(a[4], at::kInt, c->device, (int64_t)kv.n_seq + 1);
        if (!q || !cq || total_k < 0 || total_k > INT32_MAX) return decline();
        Tensor out = like(*q);
        if (!fill(out, &ro, q->size(0), c->cfg->Hq, c->cfg->d)) return decline();
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        s = lola_paged_prefill(c->cfg, &kv, (int32_t)q->size(0), (int32_t)total_k, (const int32_t*)cq->data_ptr(), &rq, &ro, nullptr,
                               c->stream.stream());
        Py_END_ALLOW_THREADS
        return s == LOLA_OK ? THPVariable_Wrap(std::move(out)) : decline();
    });
}

// decode(layer, k_pool, v_pool, q, kv_len, table) -> out
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == 6 ? begin(a[0]) : std::nullopt;
        lola_paged_kv kv;
        if (!c || !cache(a[1], a[2], a[4], a[5], *c, &kv)) return decline();
        lola_rows rq, ro;
        const Tensor* q = rows(a[3], &rq, *c, kv.n_seq, c->cfg->Hq);
        if (!q) return decline();
        Tensor out = like(*q);
        if (!fill(out, &ro, q->size(0), c->cfg->Hq, c->cfg->d)) return decline();
        // the workspace, released to torch behind the call
        const at::DataPtr ws = scratch(c->ws);
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        s = lola_paged_decode(c->cfg, &kv, &rq, &ro, nullptr, ws.get(), (size_t)c->ws, c->stream.stream());
        Py_END_ALLOW_THREADS
        return s == LOLA_OK ? THPVariable_Wrap(std::move(out)) : decline();
    });
}

// quant_pools(address of the layer's lola_attn_config, k_pool, v_pool, k_scale, v_scale) -> True where they fit the layer (and are
// on the current device)
PyObject* quant_pools(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto* cfg = n == 5 ? (const lola_attn_config*)(uintptr_t)PyLong_AsUnsignedLongLong(a[0]) : nullptr;
        if (PyErr_Occurred() || !cfg || c10::cuda::device_count() == 0) return decline();
        const int device = c10::cuda::current_device();
        lola_paged_kv kv;
        lola_kv_scales sc;
        if (!pools(a[1], a[2], device, cfg, &kv, at::kFloat8_e4m3fn) || !powers(a[3], a[4], device, cfg, kv, &sc)) return decline();
        Py_RETURN_TRUE;
    });
}

// quant_decode(layer, k_pool, v_pool, k_scale, v_scale, q, kv_len, table) -> out
PyObject* quant_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == 8 ? begin(a[0]) : std::nullopt;
        lola_paged_kv kv;
        lola_kv_scales sc;
        if (!c || !cache(a[1], a[2], a[3], a[4], a[6], a[7], *c, &kv, &sc)) return decline();
        lola_rows rq, ro;
        const Tensor* q = rows(a[5], &rq, *c, kv.n_seq, c->cfg->Hq);
        if (!q) return decline();
        Tensor out = like(*q);
        if (!fill(out, &ro, q->size(0), c->cfg->Hq, c->cfg->d)) return decline();
        const at::DataPtr ws = scratch(c->ws);
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        s = lola_quant_decode(c->cfg, &kv, &sc, &rq, &ro, nullptr, ws.get(), (size_t)c->ws, c->stream.stream());
        Py_END_ALLOW_THREADS
        return s == LOLA_OK ? THPVariable_Wrap(std::move(out)) : decline();
    });
}

// shared(layer, k_pool, v_pool, k_scale | None, v_scale | None, q, kv_len, table, prefix_len, prefix_table, cu | None) -> out
PyObject* shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == 11 ? begin(a[0]) : std::nullopt;
        if (!c) return decline();
        lola_paged_kv kv;
        lola_kv_scales sc;
        const bool quant = a[3] != Py_None;
        if (!(quant ? cache(a[1], a[2], a[3], a[4], a[6], a[7], *c, &kv, &sc) : cache(a[1], a[2], a[6], a[7], *c, &kv))) return decline();
        const Tensor *t = get(a[9], at::kInt, c->device), *cu = nullptr;
        if (!t || t->dim() != 2 || (t->stride(1) != 1 && t->size(1) != 1) || t->size(0) >= INT32_MAX || t->size(1) > INT32_MAX) return decline();
        const Tensor* len = vec(a[8], at::kInt, c->device, t->size(0));
        if (!len || (a[10] != Py_None && !(cu = vec(a[10], at::kInt, c->device, t->size(0) + 1)))) return decline();
        const lola_prefixes px{(int32_t)t->size(0), (int32_t)t->size(1), t->size(0) == 1 ? t->size(1) : t->stride(0), (const int32_t*)t->data_ptr(),
                               (const int32_t*)len->data_ptr(), cu ? (const int32_t*)cu->data_ptr() : nullptr};
        lola_rows rq, ro;
        const Tensor* q = rows(a[5], &rq, *c, kv.n_seq, c->cfg->Hq);
        if (!q) return decline();
        const int64_t size = lola_shared_decode_workspace_bytes(c->cfg, kv.n_seq);
        if (size < 0) return decline();
        Tensor out = like(*q);
        if (!fill(out, &ro, q->size(0), c->cfg->Hq, c->cfg->d)) return decline();
        const at::DataPtr ws = scratch(size);
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        s = lola_shared_decode(c->cfg, &kv, quant ? &sc : nullptr, &px, &rq, &ro, nullptr, ws.get(), (size_t)size, c->stream.stream());
        Py_END_ALLOW_THREADS
        return s == LOLA_OK ? THPVariable_Wrap(std::move(out)) : decline();
    });
}

// quant_read(layer, k_pool, v_pool, k_scale, v_scale, kv_len, table, total) -> (k, v, cu)
PyObject* quant_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == 8 ? begin(a[0]) : std::nullopt;
        lola_paged_kv kv;
        lola_kv_scales sc;
        if (!c || !cache(a[1], a[2], a[3], a[4], a[5], a[6], *c, &kv, &sc)) return decline();
        const long long total = PyLong_Check(a[7]) ? PyLong_AsLongLong(a[7]) : -1;
        if (total < 0 || total > INT32_MAX) return decline();
        Tensor k = empty({total, c->cfg->Hkv, c->cfg->d}, c->dtype, c->device), v = empty(k.sizes(), c->dtype, c->device);
        Tensor cu = empty({(int64_t)kv.n_seq + 1}, at::kInt, c->device);
        lola_rows rk, rv;
        if (!fill(k, &rk, total, c->cfg->Hkv, c->cfg->d) || !fill(v, &rv, total, c->cfg->Hkv, c->cfg->d)) return decline();
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        s = lola_quant_read(c->cfg, &kv, &sc, (int32_t)total, &rk, &rv, (int32_t*)cu.data_ptr(), c->stream.stream());
        Py_END_ALLOW_THREADS
        if (s != LOLA_OK) return decline();
        PyObject* r = PyTuple_New(3);
        if (!r) return decline();
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(k)));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(v)));
        PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(std::move(cu)));
        return r;
    });
}

// append(layer, k_pool, v_pool, k, v, kv_len, table, cu_new | None, q | None, inv_freq | None, pairs) -> q_out, and
// quant_append(layer, k_pool, v_pool, k_scale, v_scale, k, ...)
template <bool QZ> PyObject* append_to(PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        const auto c = n == (QZ ? 13 : 11) ? begin(a[0]) : std::nullopt;
        lola_paged_kv kv;
        [[maybe_unused]] lola_kv_scales sc;
        if (!c) return decline();
        if constexpr (QZ) {
            if (!cache(a[1], a[2], a[3], a[4], a[7], a[8], *c, &kv, &sc)) return decline();
            a += 2;                                        // (k and what follows it, by the other's numbers)
        } else if (!cache(a[1], a[2], a[5], a[6], *c, &kv)) {
            return decline();
        }
        const long pairs = PyLong_AsLong(a[10]);
        if (pairs == -1 && PyErr_Occurred()) return decline();
        lola_rows rk, rv, rq, ro;
        const Tensor *k = rows(a[3], &rk, *c, -1, c->cfg->Hkv), *q = nullptr, *cu = nullptr, *freq = nullptr;
        if (!k || !rows(a[4], &rv, *c, k->size(0), c->cfg->Hkv) ||
            (a[7] != Py_None && !(cu = vec(a[7], at::kInt, c->device, (int64_t)kv.n_seq + 1))) ||
            (a[8] != Py_None && !(q = rows(a[8], &rq, *c, k->size(0), c->cfg->Hq))) ||
            (a[9] != Py_None && (!(freq = vec(a[9], at::kFloat, c->device, -1)) || freq->size(0) > 1024)))
            return decline();
        Tensor out;
        if (q) {
            out = like(*q);
            if (!fill(out, &ro, q->size(0), c->cfg->Hq, c->cfg->d)) return decline();
        }
        int32_t s;
        Py_BEGIN_ALLOW_THREADS
        auto call = [&](auto f, auto... more) {
            return f(c->cfg, &kv, more..., (int32_t)k->size(0), cu ? (const int32_t*)cu->data_ptr() : nullptr, &rk, &rv, q ? &rq : nullptr,
                     q ? &ro : nullptr, freq ? (const float*)freq->data_ptr() : nullptr, freq ? (int32_t)(2 * freq->size(0)) : 0,
                     (int32_t)pairs, nullptr, c->stream.stream());
        };
        if constexpr (QZ) s = call(lola_quant_append, &sc);
        else s = call(lola_paged_append);
        Py_END_ALLOW_THREADS
        if (s != LOLA_OK) return decline();
        if (q) return THPVariable_Wrap(std::move(out));
        Py_RETURN_NONE;
    });
}

PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) { return append_to<false>(a, n); }
PyObject* quant_append(PyObject*, PyObject* const* a, Py_ssize_t n) { return append_to<true>(a, n); }

PyMethodDef methods[] = {
    {"prefill", (PyCFunction)(void (*)(void))prefill, METH_FASTCALL, nullptr},
    {"prefill_paged", (PyCFunction)(void (*)(void))prefill_paged, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"quant_pools", (PyCFunction)(void (*)(void))quant_pools, METH_FASTCALL, nullptr},
    {"quant_append", (PyCFunction)(void (*)(void))quant_append, METH_FASTCALL, nullptr},
    {"quant_decode", (PyCFunction)(void (*)(void))quant_decode, METH_FASTCALL, nullptr},
    {"quant_read", (PyCFunction)(void (*)(void))quant_read, METH_FASTCALL, nullptr},
    {"shared", (PyCFunction)(void (*)(void))shared, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lola_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lola_py(void) { return PyModule_Create(&module); }
