// Native host path of the QSA layer's Python calls.
//
// A decode step's norm, append or single-token attention takes 3 to 10 us on the GPU; checking and
// marshalling its arguments in Python took as long or longer.  These functions check a call's
// tensors, allocate its outputs and call the library's entry point, for well-formed calls on the
// current device and stream; anything else (a wrong type, another device, an error status) returns
// None, and the Python function then takes its own way, with its own errors.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>

#include "libgdn.h"

namespace {

decltype(&gdn_qsa_norm_rope) norm_rope_fn = nullptr;
decltype(&gdn_qsa_kv_append) kv_append_fn = nullptr;
decltype(&gdn_qsa_attention) attention_fn = nullptr;

// a plain tensor on `dev`, or null
const at::Tensor *tensor(PyObject *o, int64_t dev) {
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == dev ? &t : nullptr;
}
bool row_dtype(const at::Tensor &t, gdn_dtype &code) {
    if (t.scalar_type() == at::kBFloat16) code = GDN_BF16;
    else if (t.scalar_type() == at::kFloat) code = GDN_F32;
    else return false;
    return true;
}
// head rows [B, Tn, heads, d] with contiguous heads and evenly spaced tokens: elements from one to the next
bool rows(const at::Tensor &t, int64_t &step) {
    if (t.dim() != 4) return false;
    const auto n = t.sizes(), s = t.strides();
    step = n[1] > 1 ? s[1] : n[0] > 1 ? s[0] : n[2] * n[3];
    return !((n[3] > 1 && s[3] != 1) || (n[2] > 1 && s[2] != n[3]) || (n[0] > 1 && n[1] > 1 && s[0] != n[1] * s[1]));
}
// int32 [a] or [a, b], contiguous; None where `none` allows it
bool ints(PyObject *o, int64_t dev, at::IntArrayRef shape, bool none, const int32_t *&p) {
    p = nullptr;
    if (o == Py_None) return none;
    const at::Tensor *t = tensor(o, dev);
    if (!t || t->scalar_type() != at::kInt || t->sizes() != shape || !t->is_contiguous()) return false;
    p = static_cast<const int32_t *>(t->data_ptr());
    return true;
}
bool weight(PyObject *o, int64_t dev, int64_t d, const float *&p) {
    p = nullptr;
    if (o == Py_None) return true;
    const at::Tensor *t = tensor(o, dev);
    if (!t || t->scalar_type() != at::kFloat || t->dim() != 1 || t->size(0) != d || !t->is_contiguous()) return false;
    p = static_cast<const float *>(t->data_ptr());
    return true;
}
bool caches(PyObject *ko, PyObject *vo, int64_t dev, int64_t heads, int64_t d, const at::Tensor *&k, const at::Tensor *&v) {
    k = tensor(ko, dev);
    v = tensor(vo, dev);
    return k && v && k->dim() == 4 && k->scalar_type() == at::kBFloat16 && v->scalar_type() == at::kBFloat16 &&
           k->sizes() == v->sizes() && (heads < 0 || k->size(1) == heads) && k->size(3) == d && k->is_contiguous() &&
           v->is_contiguous();
}
bool small(int64_t a) { return a >= 0 && a <= INT32_MAX; }
bool real(PyObject *o, float &x) {
    if (!PyFloat_Check(o) && !PyLong_Check(o)) return false;
    x = (float)PyFloat_AsDouble(o);
    if (!PyErr_Occurred()) return true;
    PyErr_Clear();
    return false;
}
bool whole(PyObject *o, int &x) {
    if (!PyLong_Check(o)) return false;
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(o, &over);
    if (over || v < 0 || v > INT32_MAX) return false;
    x = (int)v;
    return true;
}

// (q, w_q, pos, k, w_k, rope_dim, eps, theta) -> q_out, (q_out, k_out) or None
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        const int64_t dev = c10::cuda::current_device();
        const at::Tensor *q = n == 8 ? tensor(a[0], dev) : nullptr, *k = nullptr;
        gdn_dtype code, k_code;
        int64_t q_step, k_step = 0;
        if (!norm_rope_fn || !q || !row_dtype(*q, code) || !rows(*q, q_step)) Py_RETURN_NONE;
        const int64_t B = q->size(0), T = q->size(1), hq = q->size(2), d = q->size(3);
        if (a[3] != Py_None) {
            k = tensor(a[3], dev);
            if (!k || !row_dtype(*k, k_code) || k_code != code || !rows(*k, k_step) || k->size(0) != B || k->size(1) != T ||
                k->size(3) != d)
                Py_RETURN_NONE;
        }
        const int64_t hk = k ? k->size(2) : 0;
        const int32_t *pos;
        const float *wq, *wk;
        int rope;
        float eps, theta;
        if (!small(B) || !small(T) || !small(hq) || !small(hk) || !small(d) || !ints(a[2], dev, {B}, false, pos) ||
            !weight(a[1], dev, d, wq) || !weight(a[4], dev, d, wk) || !whole(a[5], rope) || !real(a[6], eps) ||
            !real(a[7], theta))
            Py_RETURN_NONE;
        at::Tensor qo = at::detail::empty_cuda(q->sizes(), q->options()), ko;
        if (k) ko = at::detail::empty_cuda(k->sizes(), k->options());
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev);
        gdn_status st;
        Py_BEGIN_ALLOW_THREADS
        st = norm_rope_fn(q->data_ptr(), k ? k->data_ptr() : nullptr, code, q_step, k_step, wq, wk, pos, (int)B, (int)T,
                          (int)hq, (int)hk, (int)d, rope, eps, theta, qo.data_ptr(), k ? ko.data_ptr() : nullptr, code, stream);
        Py_END_ALLOW_THREADS
        if (st != GDN_OK) Py_RETURN_NONE;
        PyObject *x = THPVariable_Wrap(std::move(qo));
        if (!k || !x) return x;
        PyObject *y = THPVariable_Wrap(std::move(ko)), *r = y ? PyTuple_Pack(2, x, y) : nullptr;
        Py_DECREF(x);
        Py_XDECREF(y);
        return r;
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (k, v, w_k, pos, page_table, k_cache, v_cache, n_new, rope_dim, eps, theta) -> True or None
PyObject *kv_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        const int64_t dev = c10::cuda::current_device();
        const at::Tensor *k = n == 11 ? tensor(a[0], dev) : nullptr, *v = k ? tensor(a[1], dev) : nullptr, *kc, *vc;
        gdn_dtype code, v_code;
        int64_t k_step, v_step;
        if (!kv_append_fn || !v || !row_dtype(*k, code) || !row_dtype(*v, v_code) || code != v_code || !rows(*k, k_step) ||
            !rows(*v, v_step) || k->sizes() != v->sizes())
            Py_RETURN_NONE;
        const int64_t B = k->size(0), T = k->size(1), hk = k->size(2), d = k->size(3);
        const at::Tensor *table = tensor(a[4], dev);
        if (!table || table->dim() != 2 || !caches(a[5], a[6], dev, hk, d, kc, vc)) Py_RETURN_NONE;
        const int64_t max_pages = table->size(1);
        const int32_t *pos, *tab, *n_new;
        const float *wk;
        int rope;
        float eps, theta;
        if (!small(B) || !small(T) || !small(hk) || !small(d) || !small(max_pages) || !small(kc->size(0)) || !small(kc->size(2)) ||
            !ints(a[3], dev, {B}, false, pos) || !ints(a[4], dev, {B, max_pages}, false, tab) ||
            !ints(a[7], dev, {B}, true, n_new) || !weight(a[2], dev, d, wk) || !whole(a[8], rope) || !real(a[9], eps) ||
            !real(a[10], theta))
            Py_RETURN_NONE;
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev);
        gdn_status st;
        Py_BEGIN_ALLOW_THREADS
        st = kv_append_fn(k->data_ptr(), v->data_ptr(), code, k_step, v_step, wk, pos, n_new, (int)B, (int)T, tab,
                          (int)max_pages, (int)hk, (int)d, rope, eps, theta, kc->data_ptr(), vc->data_ptr(),
                          (int)kc->size(0), (int)kc->size(2), stream);
        Py_END_ALLOW_THREADS
        if (st != GDN_OK) Py_RETURN_NONE;
        Py_RETURN_TRUE;
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (q, blocks, qpos, page_table, k_cache, v_cache, n_query, scale or None) -> out or None
PyObject *attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    try {
        const int64_t dev = c10::cuda::current_device();
        const at::Tensor *q = n == 8 ? tensor(a[0], dev) : nullptr, *kc, *vc;
        if (!attention_fn || !q || q->scalar_type() != at::kBFloat16 || q->dim() != 4 || !q->is_contiguous()) Py_RETURN_NONE;
        const int64_t B = q->size(0), Qn = q->size(1), hq = q->size(2), d = q->size(3);
        const at::Tensor *blocks = tensor(a[1], dev), *table = tensor(a[3], dev);
        if (!blocks || blocks->dim() != 3 || !table || table->dim() != 2 || !caches(a[4], a[5], dev, -1, d, kc, vc))
            Py_RETURN_NONE;
        const int64_t slots = blocks->size(2), max_pages = table->size(1);
        const int32_t *list, *pos, *tab, *n_query;
        float scale = 0.f;
        if (a[7] == Py_None) scale = (float)std::pow((double)d, -0.5);
        else if (!real(a[7], scale)) Py_RETURN_NONE;
        if (!small(B) || !small(Qn) || !small(hq) || !small(d) || !small(slots) || !small(max_pages) || !small(kc->size(0)) ||
            !small(kc->size(1)) || !small(kc->size(2)) || !ints(a[1], dev, {B, Qn, slots}, false, list) ||
            !ints(a[2], dev, {B}, false, pos) || !ints(a[3], dev, {B, max_pages}, false, tab) ||
            !ints(a[6], dev, {B}, true, n_query))
            Py_RETURN_NONE;
        at::Tensor out = at::detail::empty_cuda(q->sizes(), q->options());
        const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev);
        gdn_status st;
        Py_BEGIN_ALLOW_THREADS
        st = attention_fn(q->data_ptr(), list, (int)slots, pos, n_query, (int)B, (int)Qn, tab, (int)max_pages, (int)hq,
                          (int)kc->size(1), (int)d, kc->data_ptr(), vc->data_ptr(), (int)kc->size(0), (int)kc->size(2), scale,
                          out.data_ptr(), stream);
        Py_END_ALLOW_THREADS
        if (st != GDN_OK) Py_RETURN_NONE;
        return THPVariable_Wrap(std::move(out));
    } catch (...) {
        Py_RETURN_NONE;
    }
}

// (addresses of the three entry points of the loaded library)
PyObject *bind(PyObject *, PyObject *args) {
    unsigned long long x, y, z;
    if (!PyArg_ParseTuple(args, "KKK", &x, &y, &z)) return nullptr;
    norm_rope_fn = reinterpret_cast<decltype(norm_rope_fn)>(x);
    kv_append_fn = reinterpret_cast<decltype(kv_append_fn)>(y);
    attention_fn = reinterpret_cast<decltype(attention_fn)>(z);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rope)), METH_FASTCALL, nullptr},
    {"kv_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kv_append)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and Python whose headers this file was compiled against
PyMODINIT_FUNC PyInit__fast() {
    PyObject *m = PyModule_Create(&module_def);
    if (m && PyModule_AddStringConstant(m, "built_for", GDN_BUILT_FOR) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
