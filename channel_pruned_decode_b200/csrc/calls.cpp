// Native half of the Python binding of the paged 8-bit cache's calls: checks
// the tensors and calls the C ABI.  A decode step makes three of these calls a
// layer, and their checks and argument conversion in Python cost more than the
// kernels of a small step (7.5 us a call; here less than the launch).
//
// Each function takes the Python function's arguments in order, then the
// stream (None: the current one), and returns the library's status, or -1
// where a tensor is not what the call needs: the caller then says which.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <limits.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "spark.h"

namespace {

constexpr long kRefused = -1;

// The tensor of a Python argument; nullptr if it is none.
const at::Tensor *tensor(PyObject *o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool fits(const at::Tensor *t, at::ScalarType type, int64_t device) {
    return t && t->scalar_type() == type && t->is_contiguous() && t->is_cuda() && t->get_device() == device;
}

// fits, with sizes that the library's int arguments hold
bool fits_int(const at::Tensor *t, int64_t device) { return fits(t, at::kInt, device) && t->numel() <= INT_MAX; }

bool row(const at::Tensor *t, int64_t n, int64_t device) { return fits_int(t, device) && t->numel() == n; }

bool matrix(const at::Tensor *t, int64_t rows, int64_t device) {
    return fits(t, at::kInt, device) && t->dim() == 2 && t->size(0) == rows && rows <= INT_MAX && t->size(1) <= INT_MAX;
}

bool shape(const at::Tensor *t, at::IntArrayRef s) { return t->sizes() == s; }

int32_t *ints(const at::Tensor *t) { return static_cast<int32_t *>(t->data_ptr()); }

// The stream to launch on; kernels start on the current device, so the
// tensors must be there.
bool stream_of(PyObject *o, int64_t device, void **stream) {
    if (device != c10::cuda::current_device()) return false;
    if (o == Py_None) {
        *stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
        return true;
    }
    *stream = PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
}

bool small_int(PyObject *o, int *x) {
    const long v = PyLong_AsLong(o);
    if ((v == -1 && PyErr_Occurred()) || v != static_cast<int>(v)) {
        PyErr_Clear();
        return false;
    }
    *x = static_cast<int>(v);
    return true;
}

int dtype_of(const at::Tensor *t) {
    return t->scalar_type() == at::kBFloat16 ? SPARK_BF16 : t->scalar_type() == at::kFloat ? SPARK_F32 : -1;
}

// lens, n_new, page, pool, taken, table, slots, lens_out, taken_out, ws, stream, n_served or None
long pages_extend(PyObject *const *a) {
    const at::Tensor *lens = tensor(a[0]), *n_new = tensor(a[1]), *pool = tensor(a[3]), *taken = tensor(a[4]),
                     *table = tensor(a[5]), *slots = tensor(a[6]), *lens_out = tensor(a[7]),
                     *taken_out = tensor(a[8]), *ws = tensor(a[9]),
                     *served = a[11] == Py_None ? nullptr : tensor(a[11]);
    int page;
    void *st;
    if (!lens || !lens->is_cuda() || !small_int(a[2], &page)) return kRefused;
    const int64_t dev = lens->get_device(), B = lens->numel();
    if (lens->dim() != 1 || !row(lens, B, dev) || !row(n_new, B, dev) || !row(lens_out, B, dev) ||
        !matrix(table, B, dev) || !matrix(slots, B, dev) || !fits_int(pool, dev) || !row(taken, 1, dev) ||
        !row(taken_out, 1, dev) || (a[11] != Py_None && !row(served, B, dev)) || !ws ||
        !fits(ws, ws->scalar_type(), dev) || !stream_of(a[10], dev, &st))
        return kRefused;
    if (served)
        return spark_pages_extend_served(ints(lens), ints(n_new), (int)B, page, ints(pool), (int)pool->numel(),
                                         ints(taken), ints(table), (int)table->size(1), (int)slots->size(1),
                                         ints(slots), ints(lens_out), ints(taken_out), ints(served), ws->data_ptr(),
                                         ws->nbytes(), st);
    return spark_pages_extend(ints(lens), ints(n_new), (int)B, page, ints(pool), (int)pool->numel(), ints(taken),
                              ints(table), (int)table->size(1), (int)slots->size(1), ints(slots), ints(lens_out),
                              ints(taken_out), ws->data_ptr(), ws->nbytes(), st);
}

// lens, keep, page, pool, taken, table, lens_out, taken_out, ws, stream
long pages_trim(PyObject *const *a) {
    const at::Tensor *lens = tensor(a[0]), *keep = tensor(a[1]), *pool = tensor(a[3]), *taken = tensor(a[4]),
                     *table = tensor(a[5]), *lens_out = tensor(a[6]), *taken_out = tensor(a[7]), *ws = tensor(a[8]);
    int page;
    void *st;
    if (!lens || !lens->is_cuda() || !small_int(a[2], &page)) return kRefused;
    const int64_t dev = lens->get_device(), B = lens->numel();
    if (lens->dim() != 1 || !row(lens, B, dev) || !row(keep, B, dev) || !row(lens_out, B, dev) ||
        !matrix(table, B, dev) || !fits_int(pool, dev) || !row(taken, 1, dev) || !row(taken_out, 1, dev) ||
        !ws || !fits(ws, ws->scalar_type(), dev) || !stream_of(a[9], dev, &st))
        return kRefused;
    return spark_pages_trim(ints(lens), ints(keep), (int)B, page, ints(pool), (int)pool->numel(), ints(taken),
                            ints(table), (int)table->size(1), ints(lens_out), ints(taken_out), ws->data_ptr(),
                            ws->nbytes(), st);
}

// k_new, v_new, slots, cache descriptor's address, cache's device, ws, stream
long kv8_append(PyObject *const *a) {
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *slots = tensor(a[2]), *ws = tensor(a[5]);
    const auto *kc = static_cast<const spark_kv8cache *>(PyLong_AsVoidPtr(a[3]));
    int dev;
    void *st;
    if (!k || !slots || !kc || !small_int(a[4], &dev) || slots->dim() != 2) return kRefused;
    const int64_t B = slots->size(0), n = slots->size(1);
    const bool flat = n == 1 && k->dim() == 3;
    const int64_t s4[4] = {B, kc->Hkv, n, kc->D}, s3[3] = {B, kc->Hkv, kc->D};
    const at::IntArrayRef want = flat ? at::IntArrayRef(s3, 3) : at::IntArrayRef(s4, 4);
    if (dtype_of(k) < 0 || !fits(k, k->scalar_type(), dev) || !fits(v, k->scalar_type(), dev) || !shape(k, want) ||
        !shape(v, want) || !matrix(slots, B, dev) || !ws || !fits(ws, ws->scalar_type(), dev) ||
        !stream_of(a[6], dev, &st))
        return kRefused;
    return spark_kv8_append(k->data_ptr(), v->data_ptr(), (int)B, (int)n, dtype_of(k), ints(slots), kc,
                            ws->data_ptr(), ws->nbytes(), st);
}

// q, cache descriptor's address, cache's device, table, lens, G, out, ws, n_new or None, stream
long decode_attn_kv8(PyObject *const *a) {
    const at::Tensor *q = tensor(a[0]), *table = tensor(a[3]), *lens = tensor(a[4]), *out = tensor(a[6]),
                     *ws = tensor(a[7]), *n_new = a[8] == Py_None ? nullptr : tensor(a[8]);
    const auto *kc = static_cast<const spark_kv8cache *>(PyLong_AsVoidPtr(a[1]));
    int dev, G;
    void *st;
    if (!q || !table || !kc || !small_int(a[2], &dev) || !small_int(a[5], &G) || table->dim() != 2) return kRefused;
    const int64_t B = table->size(0), n_q = q->dim() == 4 ? q->size(2) : 1;
    const int64_t s4[4] = {B, (int64_t)kc->Hkv * G, n_q, kc->D}, s3[3] = {B, (int64_t)kc->Hkv * G, kc->D};
    const at::IntArrayRef want = q->dim() == 4 ? at::IntArrayRef(s4, 4) : at::IntArrayRef(s3, 3);
    if (dtype_of(q) < 0 || !fits(q, q->scalar_type(), dev) || !shape(q, want) || !fits(out, at::kFloat, dev) ||
        !shape(out, want) || !matrix(table, B, dev) || !row(lens, B, dev) ||
        (a[8] != Py_None && !row(n_new, B, dev)) || !ws || !fits(ws, ws->scalar_type(), dev) ||
        !stream_of(a[9], dev, &st))
        return kRefused;
    return spark_decode_attn_kv8(q->data_ptr(), dtype_of(q), kc, ints(table), (int)table->size(1), ints(lens),
                                 n_new ? ints(n_new) : nullptr, (int)B, G, (int)n_q,
                                 static_cast<float *>(out->data_ptr()), ws->data_ptr(), ws->nbytes(), st);
}

// No C++ exception leaves through the interpreter.
template <long (*kCall)(PyObject *const *), Py_ssize_t kArgs>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%zd arguments needed, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        const long rc = kCall(args);
        return PyErr_Occurred() ? nullptr : PyLong_FromLong(rc);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

template <long (*kCall)(PyObject *const *), Py_ssize_t kArgs> PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<kCall, kArgs>)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {method<pages_extend, 12>("pages_extend"), method<pages_trim, 10>("pages_trim"),
                         method<kv8_append, 7>("kv8_append"), method<decode_attn_kv8, 10>("decode_attn_kv8"),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject *PyInit__calls() {
    PyObject *m = PyModule_Create(&module_def);
    // the binding refuses to use it under another torch or Python
    if (m && PyModule_AddStringConstant(m, "built_for", SPARK_BUILT_FOR) < 0) Py_CLEAR(m);
    return m;
}
