// Python entry of the operators around the block: checks tensors against a
// call's dims and calls the C ABI with their pointers. In Python these checks
// and the ctypes conversion cost 4 us a call, more than the kernels that a
// decode batch launches; here they cost 0.6.
//
// Every function takes the dims structure (anything with the buffer
// interface), the tensors (or None) and the stream handle, raises ValueError
// for a tensor that does not fit, and returns the library's status.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "../../include/moe_w8a8.h"

namespace {

struct Misfit {};  // a Python error is set

[[noreturn]] void refuse(const char *format, ...) {
    va_list args;
    va_start(args, format);
    PyErr_FormatV(PyExc_ValueError, format, args);
    va_end(args);
    throw Misfit{};
}

template <typename D>
D dims_of(PyObject *o) {
    Py_buffer view;
    if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw Misfit{};
    D d;
    const bool fits = view.len == static_cast<Py_ssize_t>(sizeof d);
    if (fits) memcpy(&d, view.buf, sizeof d);
    PyBuffer_Release(&view);
    if (!fits) refuse("dims: not the structure of this call");
    return d;
}

at::ScalarType type_of(int code) {
    switch (code) {
        case MOE_DTYPE_BF16: return at::kBFloat16;
        case MOE_DTYPE_FP16: return at::kHalf;
        case MOE_DTYPE_FP32: return at::kFloat;
        case MOE_DTYPE_INT8: return at::kChar;
    }
    return at::ScalarType::Undefined;
}

// The tensors of one call: all on the device of the first.
struct Tensors {
    int device = -2;
    void *get(PyObject *o, const char *name, at::ScalarType type, int64_t numel) {
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse("%s: expected a tensor or None", name);
        const at::Tensor &t = THPVariable_Unpack(o);
        if (t.scalar_type() != type || t.numel() != numel)
            refuse("%s: expected %lld elements of %s, got %lld of %s", name, static_cast<long long>(numel),
                   at::toString(type), static_cast<long long>(t.numel()), at::toString(t.scalar_type()));
        if (device == -2) device = t.is_cuda() ? t.get_device() : -1;
        if (!t.is_cuda() || t.get_device() != device)
            refuse("%s: expected a tensor on the GPU that holds the call's first tensor", name);
        if (!t.is_contiguous()) refuse("%s: tensors passed to libmoe_w8a8 must be contiguous", name);
        return t.data_ptr();
    }
};

void *handle_of(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Misfit{};
    return p;
}

// The library's call, without the interpreter's lock: a launch may wait for
// room in the queue, and what empties it for another Python thread.
template <typename F>
moe_status_t unlocked(F f) {
    PyThreadState *state = PyEval_SaveThread();
    const moe_status_t st = f();
    PyEval_RestoreThread(state);
    return st;
}

// Runs f, which may refuse; no C++ exception reaches Python.
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return PyLong_FromLong(f());
    } catch (const Misfit &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// dims, x, residual, weight, residual_out, y, q, q_scale, stream
PyObject *norm_quant(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const auto d = dims_of<moe_w8a8_norm_dims_t>(a[0]);
        const int64_t T = d.num_tokens, H = d.hidden;
        const at::ScalarType t = type_of(d.dtype);
        Tensors ts;
        void *x = ts.get(a[1], "x", t, T * H), *res = ts.get(a[2], "residual", t, T * H);
        void *w = ts.get(a[3], "weight", type_of(d.weight_dtype), H);
        void *ro = ts.get(a[4], "residual_out", t, T * H), *y = ts.get(a[5], "y", t, T * H);
        void *q = ts.get(a[6], "q", d.quant == MOE_QUANT_E4M3 ? at::kFloat8_e4m3fn : at::kChar, T * H);
        void *s = ts.get(a[7], "q_scale", at::kFloat, d.quant_group > 0 ? T * (H / d.quant_group) : T);
        void *stream = handle_of(a[8]);
        return unlocked([&] { return moe_w8a8_norm_quant(&d, x, res, w, ro, y, q, static_cast<float *>(s), stream); });
    });
}

// dims, x, weight, bias, expert_ids, expert_scales, workspace, workspace bytes, stream
PyObject *gate(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 9, [&] {
        const auto d = dims_of<moe_w8a8_gate_dims_t>(a[0]);
        const int64_t T = d.num_tokens, H = d.hidden, E = d.moe_expert_num, TK = T * d.topk;
        const long long bytes = PyLong_AsLongLong(a[7]);
        if (bytes == -1 && PyErr_Occurred()) throw Misfit{};
        Tensors ts;
        void *x = ts.get(a[1], "x", type_of(d.dtype), T * H), *w = ts.get(a[2], "weight", type_of(d.weight_dtype), E * H);
        void *b = ts.get(a[3], "bias", at::kFloat, E), *ids = ts.get(a[4], "expert_ids", at::kInt, TK);
        void *s = ts.get(a[5], "expert_scales", at::kFloat, TK), *ws = ts.get(a[6], "workspace", at::kByte, bytes);
        void *stream = handle_of(a[8]);
        return unlocked([&] {
            return moe_w8a8_gate(&d, x, w, static_cast<float *>(b), static_cast<int32_t *>(ids), static_cast<float *>(s),
                                 ws, static_cast<size_t>(bytes), stream);
        });
    });
}

// dims, x, x_scale, weight, bias, out, stream
PyObject *linear_w4(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 7, [&] {
        const auto d = dims_of<moe_w8a8_linear_w4_dims_t>(a[0]);
        const int64_t T = d.num_tokens, N = d.out_features;
        size_t packed = 0;
        const moe_status_t st = moe_w8a8_packed_w4_bytes(&d, &packed);
        if (st != MOE_OK) return st;
        Tensors ts;
        void *x = ts.get(a[1], "x", type_of(d.act_dtype), T * d.in_features);
        void *xs = ts.get(a[2], "x_scale", at::kFloat, T), *w = ts.get(a[3], "weight", at::kByte, packed);
        void *b = ts.get(a[4], "bias", at::kFloat, N);
        void *out = ts.get(a[5], "out", d.act_dtype == MOE_DTYPE_FP16 ? at::kHalf : at::kBFloat16, T * (d.gated ? N / 2 : N));
        void *stream = handle_of(a[6]);
        return unlocked(
            [&] { return moe_w8a8_linear_w4(&d, x, static_cast<float *>(xs), w, static_cast<float *>(b), out, stream); });
    });
}

PyMethodDef methods[] = {
    {"norm_quant", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_quant)), METH_FASTCALL, nullptr},
    {"gate", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gate)), METH_FASTCALL, nullptr},
    {"linear_w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(linear_w4)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycall() { return PyModule_Create(&module); }
