// mk_fast.cpp -- the binding's fast path for the serving operators: checks the
// tensors of a call and makes it, without the interpreter's attribute look-ups
// (an eager call of the smallest sizes is bound by those: 10 us through ctypes
// against 3 us of kernel).
//
// Every function returns 0 when the call was made and accepted, and anything
// else when it was not: the binding then goes through its checks again in
// Python, which name what is wrong.  Only the plain case is taken here: the
// tensors' device is current and the call goes to its current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mk.h"

namespace {

constexpr long kNotMine = -1;

const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

struct Rows {
    void *p = nullptr;
    long long stride = 0;
};

// Stride between the tokens of a [rows][heads][d] tensor whose heads are
// contiguous, -1 for any other layout.  Of a single row the row stride does not
// matter, its heads' and elements' do; of no rows nothing does.  The binding's
// other way asks this function too.
int64_t row_stride_of(const at::Tensor &t) {
    if (t.dim() != 3) return -1;
    const int64_t n = t.size(0), heads = t.size(1), d = t.size(2);
    if (n > 0 && ((d > 1 && t.stride(2) != 1) || (heads > 1 && t.stride(1) != d))) return -1;
    return n > 1 ? t.stride(0) : heads * d;
}

// A [rows][heads][d] tensor whose heads are contiguous.
bool rows(PyObject *o, at::ScalarType dt, int dev, int64_t n, int64_t heads, int64_t d, Rows &r) {
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != dt || !t->is_cuda() || t->get_device() != dev || t->dim() != 3 || t->size(0) != n ||
        t->size(1) != heads || t->size(2) != d)
        return false;
    r.stride = row_stride_of(*t);
    r.p = t->data_ptr();
    return r.stride >= 0;
}

// A contiguous vector of n; None gives a null pointer where `optional`.
bool vec(PyObject *o, at::ScalarType dt, int dev, int64_t n, bool optional, void *&p) {
    p = nullptr;
    if (o == Py_None) return optional;
    const at::Tensor *t = tensor(o);
    if (!t || t->scalar_type() != dt || !t->is_cuda() || t->get_device() != dev || t->dim() != 1 || t->size(0) != n ||
        (n > 1 && t->stride(0) != 1))
        return false;
    p = t->data_ptr();
    return true;
}

int64_t heads_of(PyObject *o) {
    const at::Tensor *t = tensor(o);
    return t && t->dim() == 3 ? t->size(1) : -1;
}
int64_t rows_of(PyObject *o) {
    const at::Tensor *t = tensor(o);
    return t && t->dim() == 3 ? t->size(0) : -1;
}

bool here(int dev) { return c10::cuda::current_device() == dev; }
mk_stream_t stream_of(int dev) { return (mk_stream_t)c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }

at::ScalarType type_of(int dtype) { return dtype == MK_BF16 ? at::kBFloat16 : at::kHalf; }

const mk_paged_kv *cache_of(PyObject *o) { return (const mk_paged_kv *)PyLong_AsVoidPtr(o); }

template <class F>
PyObject *answer(F f) {
    long st = kNotMine;
    try {
        st = f();
    } catch (...) {
    }
    if (PyErr_Occurred()) PyErr_Clear();     // an argument that is no number
    return PyLong_FromLong(st);
}

// kv_append(cache address, device, q, k, v, cu, start, theta, q_out, k_out, status)
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return answer([&]() -> long {
        if (n_args != 11) return kNotMine;
        const mk_paged_kv *kv = cache_of(a[0]);
        const int dev = (int)PyLong_AsLong(a[1]);
        const double theta = PyFloat_AsDouble(a[7]);
        if (PyErr_Occurred() || !kv || !here(dev)) return kNotMine;
        const at::ScalarType dt = type_of(kv->dtype);
        const int64_t n = rows_of(a[3]);
        Rows q, k, v, qo, ko;
        void *cu, *start, *status;
        if (n < 1 || n > 0x7fffffff || !rows(a[3], dt, dev, n, kv->n_kv_heads, kv->head_dim, k) ||
            !rows(a[4], dt, dev, n, kv->n_kv_heads, kv->head_dim, v))
            return kNotMine;
        int64_t nq = 0;
        if (a[2] != Py_None) {
            nq = heads_of(a[2]);
            if (nq < 1 || nq > 0x7fffffff || !rows(a[2], dt, dev, n, nq, kv->head_dim, q) ||
                !rows(a[8] == Py_None ? a[2] : a[8], dt, dev, n, nq, kv->head_dim, qo))
                return kNotMine;
        } else if (a[8] != Py_None)
            return kNotMine;
        if (a[9] != Py_None && !rows(a[9], dt, dev, n, kv->n_kv_heads, kv->head_dim, ko)) return kNotMine;
        if (!vec(a[5], at::kInt, dev, kv->n_seqs + 1ll, false, cu) || !vec(a[6], at::kInt, dev, kv->n_seqs, false, start) ||
            !vec(a[10], at::kInt, dev, 1, true, status))
            return kNotMine;
        return mk_kv_append(kv, (const int32_t *)cu, (const int32_t *)start, (int)n, (int)nq, q.p, q.stride, k.p, k.stride,
                            v.p, v.stride, (float)theta, qo.p, qo.stride, ko.p, ko.stride, (int32_t *)status,
                            stream_of(dev));
    });
}

// paged_attention(cache address, device, q, lens, max_len, out, workspace, scale, status)
PyObject *paged_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return answer([&]() -> long {
        if (n_args != 9) return kNotMine;
        const mk_paged_kv *kv = cache_of(a[0]);
        const int dev = (int)PyLong_AsLong(a[1]);
        const long max_len = PyLong_AsLong(a[4]);
        const double scale = PyFloat_AsDouble(a[7]);
        if (PyErr_Occurred() || !kv || !here(dev) || max_len < 0 || max_len > 0x7fffffff) return kNotMine;
        const at::ScalarType dt = type_of(kv->dtype);
        const int64_t nq = heads_of(a[2]);
        Rows q, out;
        void *lens, *status;
        const at::Tensor *ws = tensor(a[6]);
        if (nq < 1 || nq > 0x7fffffff || !rows(a[2], dt, dev, kv->n_seqs, nq, kv->head_dim, q) ||
            !rows(a[5], dt, dev, kv->n_seqs, nq, kv->head_dim, out) || !vec(a[3], at::kInt, dev, kv->n_seqs, false, lens) ||
            !vec(a[8], at::kInt, dev, 1, true, status))
            return kNotMine;
        if (!ws || !ws->is_cuda() || ws->get_device() != dev || !ws->is_contiguous()) return kNotMine;
        return mk_paged_attention(kv, (const int32_t *)lens, (int)max_len, (int)nq, q.p, q.stride, (float)scale, out.p,
                                  out.stride, ws->data_ptr(), ws->nbytes(), (int32_t *)status, stream_of(dev));
    });
}

// prompt_attention(q, k, v, cu, max_len, out, scale, status)
PyObject *prompt_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return answer([&]() -> long {
        if (n_args != 8) return kNotMine;
        const at::Tensor *tq = tensor(a[0]), *tcu = tensor(a[3]);
        const long max_len = PyLong_AsLong(a[4]);
        const double scale = PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred() || !tq || !tcu || tq->dim() != 3 || tcu->dim() != 1 || !tq->is_cuda() || max_len < 0 ||
            max_len > 0x7fffffff)
            return kNotMine;
        const int dev = tq->get_device();
        const at::ScalarType dt = tq->scalar_type();
        if ((dt != at::kBFloat16 && dt != at::kHalf) || !here(dev)) return kNotMine;
        const int64_t n = tq->size(0), nq = tq->size(1), d = tq->size(2), nkv = heads_of(a[1]), ns = tcu->size(0) - 1;
        Rows q, k, v, out;
        void *cu, *status;
        if (n < 1 || n > 0x7fffffff || nq > 0x7fffffff || nkv < 1 || nkv > 0x7fffffff || d > 0x7fffffff || ns < 1 ||
            ns > 0x7ffffffe || !rows(a[0], dt, dev, n, nq, d, q) || !rows(a[1], dt, dev, n, nkv, d, k) ||
            !rows(a[2], dt, dev, n, nkv, d, v) || !rows(a[5], dt, dev, n, nq, d, out) ||
            !vec(a[3], at::kInt, dev, ns + 1, false, cu) || !vec(a[7], at::kInt, dev, 1, true, status))
            return kNotMine;
        return mk_prompt_attention(dt == at::kBFloat16 ? MK_BF16 : MK_FP16, (int)nq, (int)nkv, (int)d, (const int32_t *)cu,
                                   (int)ns, (int)n, (int)max_len, q.p, q.stride, k.p, k.stride, v.p, v.stride,
                                   (float)scale, out.p, out.stride, (int32_t *)status, stream_of(dev));
    });
}

// sample(logits, uniform, token_out, temperature, top_k, top_p, min_p)
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
    return answer([&]() -> long {
        if (n_args != 7) return kNotMine;
        const at::Tensor *x = tensor(a[0]);
        if (!x || x->dim() != 2 || x->scalar_type() != at::kFloat || !x->is_cuda()) return kNotMine;
        const int dev = x->get_device();
        const int64_t n = x->size(0), vocab = x->size(1);
        if (!here(dev) || n < 1 || n > 0x7fffffff || vocab > 0x7fffffff || (vocab > 1 && x->stride(1) != 1)) return kNotMine;
        void *u, *token, *t, *k, *p, *m;
        if (!vec(a[1], at::kFloat, dev, n, false, u) || !vec(a[2], at::kInt, dev, n, false, token) ||
            !vec(a[3], at::kFloat, dev, n, true, t) || !vec(a[4], at::kInt, dev, n, true, k) ||
            !vec(a[5], at::kFloat, dev, n, true, p) || !vec(a[6], at::kFloat, dev, n, true, m))
            return kNotMine;
        return mk_sample((const float *)x->data_ptr(), n > 1 ? x->stride(0) : vocab, (int)n, (int)vocab, (const float *)u,
                         (const float *)t, (const int32_t *)k, (const float *)p, (const float *)m, (int32_t *)token,
                         stream_of(dev));
    });
}

// row_stride(tensor): row_stride_of
PyObject *row_stride(PyObject *, PyObject *o) {
    const at::Tensor *t = tensor(o);
    int64_t stride = -1;
    try {
        if (t) stride = row_stride_of(*t);
    } catch (...) {      // a tensor without strides
    }
    return PyLong_FromLongLong(stride);
}

PyMethodDef methods[] = {
    {"row_stride", row_stride, METH_O, nullptr},
    {"kv_append", (PyCFunction)(void *)kv_append, METH_FASTCALL, nullptr},
    {"paged_attention", (PyCFunction)(void *)paged_attention, METH_FASTCALL, nullptr},
    {"prompt_attention", (PyCFunction)(void *)prompt_attention, METH_FASTCALL, nullptr},
    {"sample", (PyCFunction)(void *)sample, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mk_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__mk_fast() { return PyModule_Create(&module); }
