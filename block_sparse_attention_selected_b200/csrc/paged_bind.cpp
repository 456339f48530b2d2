// paged_bind.cpp -- the short host path of the paged-cache calls for Python.
//
// A decode step calls them once per layer on kernels of a few microseconds, and marshalling a
// call in Python takes longer than that (about 12 us for an attention call, against 1 - 2 us
// here).  These functions take the plain case only: CUDA tensors of the current device, of the
// types and layouts that need no second look.  For anything else they return None and paged.py
// goes its own way, which names what is wrong; a status code of the C ABI is returned as an
// integer.  The C ABI's functions are handed over as addresses by init().
#include <Python.h>
#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "../../include/nsa_sel.h"

namespace {

decltype(&nsa_sel_paged_plan) plan_fn = nullptr;
decltype(&nsa_sel_paged_write_kv) write_fn = nullptr;
decltype(&nsa_sel_paged_attn_fwd) attn_fn = nullptr;
decltype(&nsa_sel_paged_sel_fwd) sel_fn = nullptr;

const at::Tensor* tensor(PyObject* o, at::ScalarType type, int64_t ndim, int64_t device) {
    if (!THPVariable_Check(o)) return nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != device || t.scalar_type() != type || t.dim() != ndim || t.numel() == 0)
        return nullptr;
    return &t;
}
const at::Tensor* packed(PyObject* o, at::ScalarType type, int64_t ndim, int64_t device) {
    const at::Tensor* t = tensor(o, type, ndim, device);
    return t && t->is_contiguous() ? t : nullptr;
}
const at::Tensor* strided(PyObject* o, at::ScalarType type, int64_t ndim, int64_t device) {
    const at::Tensor* t = tensor(o, type, ndim, device);
    return t && t->stride(-1) == 1 ? t : nullptr;
}

bool cache_arg(PyObject* ko, PyObject* vo, at::ScalarType type, int64_t device, nsa_paged_cache_t* c) {
    const at::Tensor *k = strided(ko, type, 4, device), *v = strided(vo, type, 4, device);
    if (!k || !v || k->sizes() != v->sizes() || k->strides() != v->strides()) return false;
    *c = nsa_paged_cache_t{k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), k->stride(2),
                           (int)k->size(0), (int)k->size(1), (int)k->size(2), (int)k->size(3)};
    return k->size(0) < (1ll << 31) && k->size(1) < (1ll << 31) && k->size(2) < (1ll << 31);
}

bool as_int(PyObject* o, int* to) {
    if (!PyLong_CheckExact(o)) return false;
    int over = 0;
    const long x = PyLong_AsLongAndOverflow(o, &over);
    if (over || x < INT32_MIN || x > INT32_MAX) return false;
    *to = (int)x;
    return true;
}
bool as_stream(PyObject* o, nsa_stream_t* to) {
    if (!PyLong_CheckExact(o)) return false;
    *to = reinterpret_cast<nsa_stream_t>(PyLong_AsVoidPtr(o));
    return !PyErr_Occurred();
}

int64_t row_stride(const at::Tensor& t) { return t.size(0) == 1 ? std::max(t.stride(0), t.size(1)) : t.stride(0); }

template <class F>
nsa_status_t without_gil(F f) {
    nsa_status_t s;
    Py_BEGIN_ALLOW_THREADS
    s = f();
    Py_END_ALLOW_THREADS
    return s;
}

template <class T>
T* ptr(const at::Tensor& t) { return static_cast<T*>(t.data_ptr()); }

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 4) return PyErr_Format(PyExc_TypeError, "init: four addresses");
    void* p[4];
    for (int i = 0; i < 4; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (PyErr_Occurred()) return nullptr;
    }
    plan_fn = reinterpret_cast<decltype(plan_fn)>(p[0]);
    write_fn = reinterpret_cast<decltype(write_fn)>(p[1]);
    attn_fn = reinterpret_cast<decltype(attn_fn)>(p[2]);
    sel_fn = reinterpret_cast<decltype(sel_fn)>(p[3]);
    Py_RETURN_NONE;
}

// plan(new_lens, cached_lens, free_pages, block_table, page_size, total_tokens, device, stream)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int page, T, device;
    nsa_stream_t stream;
    if (n != 8 || !as_int(a[4], &page) || !as_int(a[5], &T) || !as_int(a[6], &device) || !as_stream(a[7], &stream))
        Py_RETURN_NONE;
    const at::Tensor *add = packed(a[0], at::kInt, 1, device), *old = packed(a[1], at::kInt, 1, device),
                     *free = packed(a[2], at::kInt, 1, device), *table = strided(a[3], at::kInt, 2, device);
    if (!add || !old || !free || !table || T < 0 || old->size(0) != add->size(0) || table->size(0) != add->size(0) ||
        add->size(0) >= (1ll << 31) || free->size(0) >= (1ll << 31) || table->size(1) >= (1ll << 31))
        Py_RETURN_NONE;
    const int64_t R = add->size(0);
    const auto i32 = add->options();
    at::Tensor cu = at::empty({R + 1}, i32), kv = at::empty({R}, i32), slots = at::empty({T}, i32.dtype(at::kLong)),
               positions = at::empty({T}, i32), used = at::empty({1}, i32);
    const nsa_status_t s = without_gil([&] {
        return plan_fn(ptr<int32_t>(*add), ptr<int32_t>(*old), (int)R, ptr<int32_t>(*free), (int)free->size(0),
                       ptr<int32_t>(*table), (int)table->size(1), row_stride(*table), page, T, ptr<int32_t>(cu),
                       ptr<int32_t>(kv), ptr<int64_t>(slots), ptr<int32_t>(positions), ptr<int32_t>(used), stream);
    });
    if (s != NSA_OK) return PyLong_FromLong(s);
    return Py_BuildValue("(NNNNN)", THPVariable_Wrap(std::move(cu)), THPVariable_Wrap(std::move(kv)),
                         THPVariable_Wrap(std::move(slots)), THPVariable_Wrap(std::move(positions)),
                         THPVariable_Wrap(std::move(used)));
    END_HANDLE_TH_ERRORS
}

// write(k, v, slots, k_cache, v_cache, device, stream)
PyObject* write(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int device;
    nsa_stream_t stream;
    if (n != 7 || !as_int(a[5], &device) || !as_stream(a[6], &stream) || !THPVariable_Check(a[0])) Py_RETURN_NONE;
    const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf) Py_RETURN_NONE;
    const at::Tensor *k = strided(a[0], type, 3, device), *v = strided(a[1], type, 3, device),
                     *slots = packed(a[2], at::kLong, 1, device);
    nsa_paged_cache_t cache;
    if (!k || !v || !slots || !cache_arg(a[3], a[4], type, device, &cache) || k->sizes() != v->sizes() ||
        slots->size(0) != k->size(0) || k->size(1) != cache.hkv || k->size(2) != cache.head_dim ||
        k->size(0) >= (1ll << 31))
        Py_RETURN_NONE;
    return PyLong_FromLong(without_gil([&] {
        return write_fn(k->data_ptr(), v->data_ptr(), k->stride(0), k->stride(1), v->stride(0), v->stride(1),
                        ptr<int64_t>(*slots), (int)k->size(0), &cache, stream);
    }));
    END_HANDLE_TH_ERRORS
}

// attend(q, k_cache, v_cache, cu_seqlens, kv_lens, block_table, block_idx or None, block_size, scale or None,
//        window_size, out or None, lse or None, with_lse, workspace, device, stream)
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    int bs, window, device;
    nsa_stream_t stream;
    if (n != 16 || !as_int(a[7], &bs) || !as_int(a[9], &window) || !as_int(a[14], &device) ||
        !as_stream(a[15], &stream) || !THPVariable_Check(a[0]) || !PyBool_Check(a[12]))
        Py_RETURN_NONE;
    const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
    if (type != at::kBFloat16 && type != at::kHalf) Py_RETURN_NONE;
    const at::Tensor *q = strided(a[0], type, 3, device), *cu = packed(a[3], at::kInt, 1, device),
                     *kv = packed(a[4], at::kInt, 1, device), *table = strided(a[5], at::kInt, 2, device),
                     *ws = packed(a[13], at::kByte, 1, device);
    nsa_paged_cache_t cache;
    if (!q || !cu || !kv || !table || !ws || !cache_arg(a[1], a[2], type, device, &cache)) Py_RETURN_NONE;
    const int64_t T = q->size(0), hq = q->size(1), d = q->size(2), R = kv->size(0);
    if (cu->size(0) != R + 1 || table->size(0) != R || d != cache.head_dim || T >= (1ll << 31) || hq >= (1ll << 31) ||
        R >= (1ll << 31) || table->size(1) >= (1ll << 31))
        Py_RETURN_NONE;
    const at::Tensor* idx = nullptr;
    if (a[6] != Py_None) {
        idx = packed(a[6], at::kInt, 3, device);
        if (!idx || idx->size(0) != T || idx->size(1) != cache.hkv || idx->size(2) >= (1ll << 31)) Py_RETURN_NONE;
    }
    double scale = 1.0 / std::sqrt((double)d);
    if (a[8] != Py_None) {
        if (!PyFloat_CheckExact(a[8])) Py_RETURN_NONE;
        scale = PyFloat_AS_DOUBLE(a[8]);
    }
    at::Tensor out, lse;
    if (a[10] == Py_None) {
        out = at::empty(q->sizes(), q->options());
    } else {
        const at::Tensor* o = packed(a[10], type, 3, device);
        if (!o || o->sizes() != q->sizes()) Py_RETURN_NONE;
        out = *o;
    }
    if (a[11] != Py_None) {
        const at::Tensor* l = packed(a[11], at::kFloat, 2, device);
        if (!l || l->size(0) != hq || l->size(1) != T) Py_RETURN_NONE;
        lse = *l;
    } else if (a[12] == Py_True) {
        lse = at::empty({hq, T}, q->options().dtype(at::kFloat));
    }
    const unsigned flags = type == at::kHalf ? NSA_F16 : 0u;
    float* lse_to = lse.defined() ? ptr<float>(lse) : nullptr;
    const nsa_status_t s = without_gil([&] {
        if (idx)
            return sel_fn(q->data_ptr(), q->stride(0), q->stride(1), (int)T, (int)hq, &cache, ptr<int32_t>(*cu),
                          ptr<int32_t>(*kv), (int)R, ptr<int32_t>(*table), (int)table->size(1), row_stride(*table),
                          ptr<int32_t>(*idx), (int)idx->size(2), bs, (float)scale, window, out.data_ptr(), lse_to,
                          ws->data_ptr(), (size_t)ws->numel(), stream, flags);
        return attn_fn(q->data_ptr(), q->stride(0), q->stride(1), (int)T, (int)hq, &cache, ptr<int32_t>(*cu),
                       ptr<int32_t>(*kv), (int)R, ptr<int32_t>(*table), (int)table->size(1), row_stride(*table),
                       (float)scale, window, out.data_ptr(), lse_to, ws->data_ptr(), (size_t)ws->numel(), stream,
                       flags);
    });
    if (s != NSA_OK) return PyLong_FromLong(s);
    PyObject *o, *l;
    if (a[10] == Py_None) o = THPVariable_Wrap(std::move(out)); else { o = a[10]; Py_INCREF(o); }
    if (a[11] != Py_None) { l = a[11]; Py_INCREF(l); }
    else if (lse.defined()) l = THPVariable_Wrap(std::move(lse));
    else { l = Py_None; Py_INCREF(l); }
    return Py_BuildValue("(NN)", o, l);
    END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(init), METH_FASTCALL, nullptr},
    {"plan", reinterpret_cast<PyCFunction>(plan), METH_FASTCALL, nullptr},
    {"write", reinterpret_cast<PyCFunction>(write), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(attend), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged_bind", nullptr, -1, methods};

}  // namespace

// built_for: the Python and torch whose layouts are compiled in
PyMODINIT_FUNC PyInit__paged_bind() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "built_for", NSA_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
