// Argument marshalling of ExactAttention's calls in C: a call from Python spends 8-10 us of the host's
// time on attribute lookups, ctypes structures and checks, more than the GPU's for a single token.
// Each function takes the tensors as they are, reads what lola.h asks for and makes the call on torch's
// current stream.  Whatever it does not take for granted -- a tensor of another shape, type or device, a
// stream, a refusal by the library -- makes it return NotImplemented with nothing enqueued: the
// Python form of the same call then says what is wrong, or handles it.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "lola.h"

namespace {

PyObject *s_shape, *s_dtype, *s_stride, *s_data_ptr, *s_get_device;          // interned names
PyObject *f_empty_like, *f_empty, *f_stream, *f_device, *t_int32, *t_float32, *t_uint8, *k_names;

struct Tensor {
    int nd, device;
    int64_t n[4], stride[4];
    void* data;
    PyObject* dtype;     // (types are single objects: compared by address, not owned)
};

bool ints(PyObject* t, int64_t* out, int* count) {
    if (!t || !PyTuple_Check(t)) return false;
    const Py_ssize_t n = PyTuple_GET_SIZE(t);
    if (n > 4) return false;
    for (Py_ssize_t i = 0; i < n; ++i) {
        out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
        if (out[i] == -1 && PyErr_Occurred()) return false;
    }
    *count = (int)n;
    return true;
}

bool number(PyObject* owned, int64_t* out) {
    if (!owned) return false;
    *out = (int64_t)PyLong_AsUnsignedLongLongMask(owned);
    Py_DECREF(owned);
    return !PyErr_Occurred();
}

bool get(PyObject* t, Tensor* o) {
    PyObject* x = PyObject_GetAttr(t, s_shape);
    bool ok = ints(x, o->n, &o->nd);
    Py_XDECREF(x);
    if (!ok) return false;
    int strides = 0;
    x = PyObject_CallMethodNoArgs(t, s_stride);
    ok = ints(x, o->stride, &strides) && strides == o->nd;
    Py_XDECREF(x);
    if (!ok) return false;
    o->dtype = PyObject_GetAttr(t, s_dtype);
    if (!o->dtype) return false;
    Py_DECREF(o->dtype);
    int64_t v;
    if (!number(PyObject_CallMethodNoArgs(t, s_data_ptr), &v)) return false;
    o->data = (void*)(uintptr_t)v;
    if (!number(PyObject_CallMethodNoArgs(t, s_get_device), &v)) return false;
    o->device = (int)(int32_t)v;
    return true;
}

// a contiguous vector of n entries (n < 0: any number)
bool vec(PyObject* t, Tensor* o, PyObject* dtype, int device, int64_t n) {
    return get(t, o) && o->nd == 1 && o->dtype == dtype && o->device == device && (n < 0 || o->n[0] == n) &&
           (o->stride[0] == 1 || o->n[0] <= 1);
}

// [n, heads, d] rows (n < 0: any number)
bool rows(PyObject* t, Tensor* o, lola_rows* r, PyObject* dtype, int device, int64_t n, int64_t heads, int64_t d) {
    if (!get(t, o) || o->nd != 3 || o->dtype != dtype || o->device != device || (n >= 0 && o->n[0] != n) ||
        o->n[1] != heads || o->n[2] != d || o->stride[2] != 1)
        return false;
    r->data = o->data;
    r->head = heads == 1 ? d : o->stride[1];
    r->row = o->n[0] == 1 ? heads * r->head : o->stride[0];
    return true;
}

// A layer as ExactAttention keeps it: (address of its lola_attn_config, its dtype, workspace bytes)
struct Layer {
    const lola_attn_config* cfg;
    PyObject* dtype;
    int64_t ws;
};
bool layer(PyObject* t, Layer* o) {
    if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != 3) return false;
    o->cfg = (const lola_attn_config*)(uintptr_t)PyLong_AsUnsignedLongLong(PyTuple_GET_ITEM(t, 0));
    o->dtype = PyTuple_GET_ITEM(t, 1);
    o->ws = PyLong_AsLongLong(PyTuple_GET_ITEM(t, 2));
    return !PyErr_Occurred();
}

bool current(int* device, void** stream) {
    int64_t v;
    if (!number(PyObject_CallNoArgs(f_device), &v)) return false;
    *device = (int)v;
    PyObject* i = PyLong_FromLong(*device);
    if (!i) return false;
    PyObject* s = PyObject_CallOneArg(f_stream, i);
    Py_DECREF(i);
    if (!number(s, &v)) return false;
    *stream = (void*)(uintptr_t)v;
    return true;
}

// a fresh output like q (owned), and its rows
PyObject* out_like(PyObject* q, lola_rows* r, const Layer& l, int device, int64_t n) {
    PyObject* out = PyObject_CallOneArg(f_empty_like, q);
    Tensor t;
    if (out && rows(out, &t, r, l.dtype, device, n, l.cfg->Hq, l.cfg->d)) return out;
    Py_XDECREF(out);
    return nullptr;
}

PyObject* decline() {
    PyErr_Clear();
    Py_RETURN_NOTIMPLEMENTED;
}

bool cache(PyObject* k_pool, PyObject* v_pool, PyObject* kv_len, PyObject* table, const Layer& l, int device, lola_paged_kv* kv) {
    Tensor k, v, n, t;
    if (k_pool == Py_None || !get(k_pool, &k) || !get(v_pool, &v) || k.nd != 4 || k.device != device || v.device != device)
        return false;
    if (!get(table, &t) || t.nd != 2 || t.dtype != t_int32 || t.device != device || (t.stride[1] != 1 && t.n[1] != 1)) return false;
    if (!vec(kv_len, &n, t_int32, device, t.n[0])) return false;
    if (k.n[0] > INT32_MAX || t.n[0] > INT32_MAX || t.n[1] > INT32_MAX) return false;
    kv->K = k.data;
    kv->V = v.data;
    kv->n_pages = (int32_t)k.n[0];
    kv->page = (int32_t)k.n[2];
    kv->n_seq = (int32_t)t.n[0];
    kv->width = (int32_t)t.n[1];
    kv->table_stride = t.n[0] == 1 ? t.n[1] : t.stride[0];
    kv->table = (const int32_t*)t.data;
    kv->kv_len = (const int32_t*)n.data;
    return true;
}

// prefill(layer, q, k, v, cu_q, cu_k | None) -> out
PyObject* prefill(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Layer l;
    int dev;
    void* st;
    Tensor q, k, v, cq, ck;
    lola_rows rq, rk, rv, ro;
    if (n != 6 || !layer(a[0], &l) || !current(&dev, &st)) return decline();
    const int64_t Hkv = l.cfg->Hkv, d = l.cfg->d;
    if (!rows(a[1], &q, &rq, l.dtype, dev, -1, l.cfg->Hq, d) || !rows(a[2], &k, &rk, l.dtype, dev, -1, Hkv, d) ||
        !rows(a[3], &v, &rv, l.dtype, dev, k.n[0], Hkv, d) || !vec(a[4], &cq, t_int32, dev, -1) ||
        (a[5] != Py_None && !vec(a[5], &ck, t_int32, dev, cq.n[0])) || q.n[0] > INT32_MAX || k.n[0] > INT32_MAX ||
        cq.n[0] > INT32_MAX)
        return decline();
    PyObject* out = out_like(a[1], &ro, l, dev, q.n[0]);
    if (!out) return decline();
    int32_t s;
    Py_BEGIN_ALLOW_THREADS
    s = lola_attn_prefill(l.cfg, (int32_t)cq.n[0] - 1, (int32_t)q.n[0], (int32_t)k.n[0], (const int32_t*)cq.data,
                          a[5] == Py_None ? nullptr : (const int32_t*)ck.data, &rq, &rk, &rv, &ro, nullptr, st);
    Py_END_ALLOW_THREADS
    if (s == LOLA_OK) return out;
    Py_DECREF(out);
    return decline();
}

// prefill_paged(layer, k_pool, v_pool, q, cu_q, kv_len, table, total_k) -> out
PyObject* prefill_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Layer l;
    int dev;
    void* st;
    Tensor q, cq;
    lola_rows rq, ro;
    lola_paged_kv kv;
    if (n != 8 || !layer(a[0], &l) || !current(&dev, &st) || !cache(a[1], a[2], a[5], a[6], l, dev, &kv)) return decline();
    const long long total_k = PyLong_Check(a[7]) ? PyLong_AsLongLong(a[7]) : -1;
    if (total_k < 0 || total_k > INT32_MAX || !rows(a[3], &q, &rq, l.dtype, dev, -1, l.cfg->Hq, l.cfg->d) || q.n[0] > INT32_MAX ||
        !vec(a[4], &cq, t_int32, dev, (int64_t)kv.n_seq + 1))
        return decline();
    PyObject* out = out_like(a[3], &ro, l, dev, q.n[0]);
    if (!out) return decline();
    int32_t s;
    Py_BEGIN_ALLOW_THREADS
    s = lola_paged_prefill(l.cfg, &kv, (int32_t)q.n[0], (int32_t)total_k, (const int32_t*)cq.data, &rq, &ro, nullptr, st);
    Py_END_ALLOW_THREADS
    if (s == LOLA_OK) return out;
    Py_DECREF(out);
    return decline();
}

// decode(layer, k_pool, v_pool, q, kv_len, table) -> out
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Layer l;
    int dev;
    void* st;
    Tensor q, w;
    lola_rows rq, ro;
    lola_paged_kv kv;
    if (n != 6 || !layer(a[0], &l) || !current(&dev, &st) || !cache(a[1], a[2], a[4], a[5], l, dev, &kv) ||
        !rows(a[3], &q, &rq, l.dtype, dev, kv.n_seq, l.cfg->Hq, l.cfg->d))
        return decline();
    PyObject* out = out_like(a[3], &ro, l, dev, kv.n_seq);
    if (!out) return decline();
    // the workspace: torch.empty(bytes, dtype=uint8, device=index), released to torch behind the call
    PyObject* args[3] = {PyLong_FromLongLong(l.ws), t_uint8, PyLong_FromLong(dev)};
    PyObject* ws = args[0] && args[2] ? PyObject_Vectorcall(f_empty, args, 1, k_names) : nullptr;
    Py_XDECREF(args[0]);
    Py_XDECREF(args[2]);
    int32_t s = LOLA_ERR_INVALID_ARG;
    if (ws && get(ws, &w)) {
        Py_BEGIN_ALLOW_THREADS
        s = lola_paged_decode(l.cfg, &kv, &rq, &ro, nullptr, w.data, (size_t)l.ws, st);
        Py_END_ALLOW_THREADS
    }
    Py_XDECREF(ws);
    if (s == LOLA_OK) return out;
    Py_DECREF(out);
    return decline();
}

// append(layer, k_pool, v_pool, k, v, kv_len, table, cu_new | None, q | None, inv_freq | None, pairs) -> q_out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    Layer l;
    int dev;
    void* st;
    Tensor k, v, q, cu, fr;
    lola_rows rk, rv, rq, ro;
    lola_paged_kv kv;
    if (n != 11 || !layer(a[0], &l) || !current(&dev, &st) || !cache(a[1], a[2], a[5], a[6], l, dev, &kv)) return decline();
    const int64_t Hkv = l.cfg->Hkv, d = l.cfg->d;
    const long pairs = PyLong_AsLong(a[10]);
    if ((pairs == -1 && PyErr_Occurred()) || !rows(a[3], &k, &rk, l.dtype, dev, -1, Hkv, d) ||
        !rows(a[4], &v, &rv, l.dtype, dev, k.n[0], Hkv, d) || k.n[0] > INT32_MAX ||
        (a[7] != Py_None && !vec(a[7], &cu, t_int32, dev, (int64_t)kv.n_seq + 1)) ||
        (a[9] != Py_None && (!vec(a[9], &fr, t_float32, dev, -1) || fr.n[0] > 1024)) ||
        (a[8] != Py_None && !rows(a[8], &q, &rq, l.dtype, dev, k.n[0], l.cfg->Hq, d)))
        return decline();
    PyObject* out = nullptr;
    if (a[8] != Py_None) {
        out = out_like(a[8], &ro, l, dev, k.n[0]);
        if (!out) return decline();
    }
    int32_t s;
    Py_BEGIN_ALLOW_THREADS
    s = lola_paged_append(l.cfg, &kv, (int32_t)k.n[0], a[7] == Py_None ? nullptr : (const int32_t*)cu.data, &rk, &rv,
                          out ? &rq : nullptr, out ? &ro : nullptr, a[9] == Py_None ? nullptr : (const float*)fr.data,
                          a[9] == Py_None ? 0 : (int32_t)(2 * fr.n[0]), (int32_t)pairs, nullptr, st);
    Py_END_ALLOW_THREADS
    if (s == LOLA_OK) {
        if (out) return out;
        Py_RETURN_NONE;
    }
    Py_XDECREF(out);
    return decline();
}

// setup(empty_like, empty, raw_stream, current_device, int32, float32, uint8)
PyObject* setup(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 7) {
        PyErr_SetString(PyExc_TypeError, "setup takes 7 arguments");
        return nullptr;
    }
    PyObject** to[] = {&f_empty_like, &f_empty, &f_stream, &f_device, &t_int32, &t_float32, &t_uint8};
    for (int i = 0; i < 7; ++i) {
        Py_INCREF(a[i]);
        Py_XSETREF(*to[i], a[i]);
    }
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"setup", (PyCFunction)(void (*)(void))setup, METH_FASTCALL, nullptr},
    {"prefill", (PyCFunction)(void (*)(void))prefill, METH_FASTCALL, nullptr},
    {"prefill_paged", (PyCFunction)(void (*)(void))prefill_paged, METH_FASTCALL, nullptr},
    {"decode", (PyCFunction)(void (*)(void))decode, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_lola_py", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lola_py(void) {
    s_shape = PyUnicode_InternFromString("shape");
    s_dtype = PyUnicode_InternFromString("dtype");
    s_stride = PyUnicode_InternFromString("stride");
    s_data_ptr = PyUnicode_InternFromString("data_ptr");
    s_get_device = PyUnicode_InternFromString("get_device");
    k_names = Py_BuildValue("(ss)", "dtype", "device");
    if (!s_shape || !s_dtype || !s_stride || !s_data_ptr || !s_get_device || !k_names) return nullptr;
    return PyModule_Create(&module);
}
