// marshal.cpp -- the binding's way into the library for calls that are shorter than
// Python takes to look at their tensors: each function checks the tensors' type, device,
// shape and layout, and calls the entry point of libarfuse that it is named after with
// their addresses.  It returns the call's status, or None, with nothing called, if a tensor
// is not what the call takes: the binding then finds out which, and says so.
//
// (An ar_rmsnorm_q8 of eight partials: 11.8 us in Python and ctypes, 3.6 us of GPU time.)
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>

#include "arfuse.h"

namespace {

decltype(&ar_rmsnorm_q8) g_rmsnorm_q8;
decltype(&ar_attn_append) g_attn_append;
decltype(&ar_attn_decode) g_attn_decode;

constexpr long kAnywhere = -2;  // device of a dry run's tensors

bool located(const at::TensorBase& t, at::ScalarType type, long device) {
    return t.scalar_type() == type && t.layout() == at::kStrided && (device == kAnywhere || (t.is_cuda() && t.get_device() == device));
}

// A contiguous tensor of this type, device and shape; its address.
bool takes(PyObject* o, at::ScalarType type, long device, std::initializer_list<int64_t> shape, void** p) {
    if (!THPVariable_Check(o)) return false;
    const at::TensorBase& t = THPVariable_Unpack(o);
    if (!located(t, type, device) || t.dim() != (int64_t)shape.size() || !t.is_contiguous()) return false;
    int64_t i = 0;
    for (const int64_t n : shape)
        if (t.size(i++) != n) return false;
    *p = t.data_ptr();
    return true;
}

bool size_of(PyObject* o, int64_t* n) {  // of the first dimension
    if (!THPVariable_Check(o)) return false;
    const at::TensorBase& t = THPVariable_Unpack(o);
    if (t.dim() < 1) return false;
    *n = t.size(0);
    return true;
}

void* address(PyObject* o) { return o == Py_None ? nullptr : PyLong_AsVoidPtr(o); }

PyObject* status(ar_status st) { return PyLong_FromLong(st); }

PyObject* none() { Py_RETURN_NONE; }

// rmsnorm_q8(handle, R, H, device, partials, residual, gamma, weight_bias, eps, group, q, scales, out or None, residual_out,
//            fp32, stream)
PyObject* rmsnorm_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 16) return PyErr_Format(PyExc_TypeError, "rmsnorm_q8 takes 16 arguments");
    const long R = PyLong_AsLong(a[1]), H = PyLong_AsLong(a[2]), device = PyLong_AsLong(a[3]), group = PyLong_AsLong(a[9]);
    const double bias = PyFloat_AsDouble(a[7]), eps = PyFloat_AsDouble(a[8]);
    const int fp32 = PyObject_IsTrue(a[14]);
    void *handle = address(a[0]), *stream = address(a[15]);
    if (PyErr_Occurred()) return nullptr;
    int64_t T;
    if (!size_of(a[5], &T) || !PyList_Check(a[4]) || PyList_GET_SIZE(a[4]) != R || R < 1 || R > AR_MAX_RANKS || group < 0) return none();
    const void* partials[AR_MAX_RANKS];
    void *p, *residual, *gamma, *q, *scales, *out = nullptr, *residual_out;
    for (long r = 0; r < R; ++r) {
        if (!takes(PyList_GET_ITEM(a[4], r), at::kBFloat16, device, {T, H}, &p)) return none();
        partials[r] = p;
    }
    if (!takes(a[5], at::kBFloat16, device, {T, H}, &residual) || !takes(a[6], at::kBFloat16, device, {H}, &gamma) ||
        !takes(a[10], at::kFloat8_e4m3fn, device, {T, H}, &q) ||
        !takes(a[11], at::kFloat, device, {T, group ? (H + group - 1) / group : 1}, &scales) ||
        (a[12] != Py_None && !takes(a[12], at::kBFloat16, device, {T, H}, &out)) ||
        !takes(a[13], fp32 ? at::kFloat : at::kBFloat16, device, {T, H}, &residual_out))
        return none();
    ar_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_rmsnorm_q8(static_cast<ar_workspace*>(handle), partials, (int)R, residual, gamma, (float)bias, (float)eps, T, (int)H, (int)group, q,
                      static_cast<float*>(scales), out, residual_out, fp32, stream);
    Py_END_ALLOW_THREADS;
    return status(st);
}

// attn_append(handle, cache, device, heads, cols of qkv, head_dim, axes, qkv, positions, slots, q, stream)
PyObject* attn_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 12) return PyErr_Format(PyExc_TypeError, "attn_append takes 12 arguments");
    const long device = PyLong_AsLong(a[2]), heads = PyLong_AsLong(a[3]), cols = PyLong_AsLong(a[4]), dim = PyLong_AsLong(a[5]),
               axes = PyLong_AsLong(a[6]);
    void *handle = address(a[0]), *cache = address(a[1]), *stream = address(a[11]);
    if (PyErr_Occurred()) return nullptr;
    int64_t T;
    void *qkv, *positions = nullptr, *slots, *q;
    if (!size_of(a[7], &T) || !takes(a[7], at::kBFloat16, device, {T, cols}, &qkv) ||
        (axes > 0 && !takes(a[8], at::kInt, device, {axes, T}, &positions) && !(axes == 1 && takes(a[8], at::kInt, device, {T}, &positions))) ||
        !takes(a[9], at::kInt, device, {T}, &slots) || !takes(a[10], at::kBFloat16, device, {T, heads, dim}, &q))
        return none();
    ar_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_attn_append(static_cast<ar_attn*>(handle), static_cast<const ar_kv_cache*>(cache), qkv, static_cast<const int32_t*>(positions),
                       static_cast<const int32_t*>(slots), T, q, stream);
    Py_END_ALLOW_THREADS;
    return status(st);
}

// attn_decode(handle, cache, device, heads, head_dim, q, page_table, lengths, scale, window, out, lse or None, stream)
PyObject* attn_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 13) return PyErr_Format(PyExc_TypeError, "attn_decode takes 13 arguments");
    const long device = PyLong_AsLong(a[2]), heads = PyLong_AsLong(a[3]), dim = PyLong_AsLong(a[4]);
    const double scale = PyFloat_AsDouble(a[8]);
    const long long window = PyLong_AsLongLong(a[9]);
    void *handle = address(a[0]), *cache = address(a[1]), *stream = address(a[12]);
    if (PyErr_Occurred()) return nullptr;
    int64_t B;
    void *q, *lengths, *out, *lse = nullptr;
    if (!size_of(a[5], &B) || !takes(a[5], at::kBFloat16, device, {B, heads, dim}, &q) || !takes(a[7], at::kInt, device, {B}, &lengths) ||
        !takes(a[10], at::kBFloat16, device, {B, heads, dim}, &out) ||
        (a[11] != Py_None && !takes(a[11], at::kFloat, device, {B, heads}, &lse)) || !THPVariable_Check(a[6]))
        return none();
    // rows of the page table may be further apart than they are long
    const at::TensorBase& table = THPVariable_Unpack(a[6]);
    if (!located(table, at::kInt, device) || table.dim() != 2 || table.size(0) != B) return none();
    const int64_t width = table.size(1), apart = B > 1 && width > 0 ? table.stride(0) : width;
    if (apart < width || (width > 1 && table.stride(1) != 1)) return none();
    const int32_t* pages = width > 0 ? static_cast<const int32_t*>(table.data_ptr()) : nullptr;
    ar_status st;
    Py_BEGIN_ALLOW_THREADS;
    st = g_attn_decode(static_cast<ar_attn*>(handle), static_cast<const ar_kv_cache*>(cache), q, pages, width, apart,
                       static_cast<const int32_t*>(lengths), B, window, (float)scale, out, static_cast<float*>(lse), stream);
    Py_END_ALLOW_THREADS;
    return status(st);
}

// bind(addresses of ar_rmsnorm_q8, ar_attn_append, ar_attn_decode): the library that was loaded
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != 3) return PyErr_Format(PyExc_TypeError, "bind takes 3 arguments");
    g_rmsnorm_q8 = reinterpret_cast<decltype(g_rmsnorm_q8)>(address(a[0]));
    g_attn_append = reinterpret_cast<decltype(g_attn_append)>(address(a[1]));
    g_attn_decode = reinterpret_cast<decltype(g_attn_decode)>(address(a[2]));
    if (PyErr_Occurred()) return nullptr;
    return none();
}

// Tensors without plain sizes or memory (nested ones, those of traces) throw when they are asked: they are not what a call
// takes either.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) noexcept {
    try {
        return F(self, a, n);
    } catch (...) {
        return none();
    }
}

PyMethodDef g_methods[] = {
    {"bind", (PyCFunction)(void*)bind, METH_FASTCALL, nullptr},
    {"rmsnorm_q8", (PyCFunction)(void*)guarded<rmsnorm_q8>, METH_FASTCALL, nullptr},
    {"attn_append", (PyCFunction)(void*)guarded<attn_append>, METH_FASTCALL, nullptr},
    {"attn_decode", (PyCFunction)(void*)guarded<attn_decode>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
