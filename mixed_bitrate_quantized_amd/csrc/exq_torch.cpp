// KVCache's calls on PyTorch tensors (the module _exq_torch): checks of shapes,
// types, strides and devices, outputs where none are given, and the call of
// the library's C entry point.  Argument marshalling only, in C++ because a
// call of a few microseconds on the GPU should not wait for more of them on
// the host: through ctypes, attention of one token took 8.9 us a call there.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <cstdarg>
#include <cstdio>
#include <exception>

#include "../../include/exq.h"

namespace {

PyObject* g_error = nullptr;   // ExqError(status, what, detail)

PyObject* raise(exq_status status, const char* what, const char* detail) {
    if (!g_error) {
        PyErr_SetString(PyExc_RuntimeError, detail);
        return nullptr;
    }
    if (PyObject* e = PyObject_CallFunction(g_error, "iss", (int)status, what, detail)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    return nullptr;
}

PyObject* refuse(const char* fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof(text), fmt, ap);
    va_end(ap);
    return raise(EXQ_ERR_INVALID_ARG, "argument check", text);
}

PyObject* status_or(exq_status st, const char* what, THPObjectPtr value) {
    return st == EXQ_OK ? value.release() : raise(st, what, exq_last_error());
}

// The arguments every call starts with: what KVCache keeps, and the stream.
struct Call {
    exq_cache_t cache;
    int64_t kv_heads, dim;
    int index;   // of the device
    void* stream;
};

bool parse(PyObject* const* a, Call& c) {
    c.cache = a[0] == Py_None ? nullptr : static_cast<exq_cache_t>(PyLong_AsVoidPtr(a[0]));
    c.kv_heads = PyLong_AsLongLong(a[1]);
    c.dim = PyLong_AsLongLong(a[2]);
    c.index = (int)PyLong_AsLong(a[3]);
    c.stream = PyLong_AsVoidPtr(a[4]);
    return !PyErr_Occurred();
}

const at::Tensor* tensor(const char* name, PyObject* o) {
    if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
    refuse("%s must be a tensor", name);
    return nullptr;
}

bool here(const at::Tensor& t, const Call& c, at::ScalarType type) {
    return t.scalar_type() == type && t.is_cuda() && t.get_device() == c.index;
}

// An fp16 operand [rows][heads][dim] with contiguous channels.
struct Rows {
    void* p;
    int64_t row, head;
};
bool rows_operand(const char* name, PyObject* o, const Call& c, int64_t rows, int64_t heads, Rows& r) {
    const at::Tensor* t = tensor(name, o);
    if (!t) return false;
    if (!here(*t, c, at::kHalf) || t->dim() != 3 || t->size(0) != rows || t->size(1) != heads || t->size(2) != c.dim ||
        t->stride(2) != 1) {
        refuse("%s must be fp16 [%lld][%lld][%lld] on cuda:%d with contiguous channels", name, (long long)rows,
               (long long)heads, (long long)c.dim, c.index);
        return false;
    }
    r = Rows{t->data_ptr(), t->stride(0), t->stride(1)};
    return true;
}

// An int32 vector of `rows`.
bool index_operand(const char* name, PyObject* o, const Call& c, int64_t rows, const int32_t*& p) {
    const at::Tensor* t = tensor(name, o);
    if (!t) return false;
    if (!here(*t, c, at::kInt) || t->dim() != 1 || t->size(0) != rows || (rows > 1 && t->stride(0) != 1)) {
        refuse("%s must be contiguous int32 [%lld] on cuda:%d", name, (long long)rows, c.index);
        return false;
    }
    p = static_cast<const int32_t*>(t->data_ptr());
    return true;
}

struct Table {
    const int32_t* p;
    int rows, width;
    int64_t stride;
};
bool table_operand(PyObject* o, const Call& c, Table& t) {
    const at::Tensor* x = tensor("table", o);
    if (!x) return false;
    if (!here(*x, c, at::kInt) || x->dim() != 2 || (x->size(1) > 1 && x->stride(1) != 1) || x->size(0) > INT32_MAX ||
        x->size(1) > INT32_MAX) {
        refuse("table must be int32 [sequences][pages] on cuda:%d with contiguous rows", c.index);
        return false;
    }
    t = Table{static_cast<const int32_t*>(x->data_ptr()), (int)x->size(0), (int)x->size(1), x->stride(0)};
    return true;
}

bool few_enough(int64_t rows) {
    if (rows <= INT32_MAX) return true;
    refuse("%lld rows", (long long)rows);
    return false;
}

at::Tensor empty(const Call& c, at::IntArrayRef shape, at::ScalarType type) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)c.index)));
}

// C++ exceptions (of PyTorch: out of memory, a tensor without storage) become
// the Python exceptions that PyTorch raises for them.
template <class F> PyObject* guarded(F&& f) {
    try {
        return f();
    } catch (...) {
        if (!PyErr_Occurred()) torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd wanted", n, want);
    return false;
}

// append(cache, kv_heads, dim, device, stream, k, v, table, seqs, positions)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c;
        if (!arity(n, 10) || !parse(a, c)) return nullptr;
        const at::Tensor* kt = tensor("k", a[5]);
        if (!kt) return nullptr;
        if (kt->dim() < 1) return refuse("k must be [rows][kv_heads][head_dim]");
        const int64_t rows = kt->size(0);
        Rows k, v;
        Table t;
        const int32_t *seqs, *positions;
        if (!few_enough(rows) || !rows_operand("k", a[5], c, rows, c.kv_heads, k) ||
            !rows_operand("v", a[6], c, rows, c.kv_heads, v) || !table_operand(a[7], c, t) ||
            !index_operand("seqs", a[8], c, rows, seqs) || !index_operand("positions", a[9], c, rows, positions))
            return nullptr;
        return status_or(exq_cache_append(c.cache, k.p, k.row, k.head, v.p, v.row, v.head, (int)rows, t.p, t.rows, t.width,
                                          t.stride, seqs, positions, c.stream),
                         "exq_cache_append", THPObjectPtr(Py_NewRef(Py_None)));
    });
}

// read(cache, kv_heads, dim, device, stream, table, seqs, positions, k_out or None, v_out or None) -> (k, v)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c;
        if (!arity(n, 10) || !parse(a, c)) return nullptr;
        const at::Tensor* st = tensor("seqs", a[6]);
        if (!st) return nullptr;
        if (st->dim() != 1) return refuse("seqs must be int32 [rows]");
        const int64_t rows = st->size(0);
        Table t;
        const int32_t *seqs, *positions;
        if (!few_enough(rows) || !table_operand(a[5], c, t) || !index_operand("seqs", a[6], c, rows, seqs) ||
            !index_operand("positions", a[7], c, rows, positions))
            return nullptr;
        THPObjectPtr out[2];
        Rows r[2];
        for (int i = 0; i < 2; ++i) {
            out[i] = a[8 + i] == Py_None ? THPVariable_Wrap(empty(c, {rows, c.kv_heads, c.dim}, at::kHalf)) : Py_NewRef(a[8 + i]);
            if (!out[i] || !rows_operand(i ? "v_out" : "k_out", out[i], c, rows, c.kv_heads, r[i])) return nullptr;
        }
        THPObjectPtr outs(PyTuple_Pack(2, out[0].get(), out[1].get()));
        if (!outs) return nullptr;
        return status_or(exq_cache_read(c.cache, r[0].p, r[0].row, r[0].head, r[1].p, r[1].row, r[1].head, (int)rows, t.p, t.rows,
                                        t.width, t.stride, seqs, positions, c.stream),
                         "exq_cache_read", std::move(outs));
    });
}

// attend(cache, kv_heads, dim, device, stream, q, table, lengths, scale, window, out or None, return_lse, lse or None,
//        workspace or None, kept workspace or None) -> out, (out, lse), or the bytes of the workspace that is missing
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        Call c;
        if (!arity(n, 15) || !parse(a, c)) return nullptr;
        const at::Tensor* qt = tensor("q", a[5]);
        if (!qt) return nullptr;
        if (qt->dim() != 3) return refuse("q must be [rows][q_heads][head_dim]");
        const int64_t rows = qt->size(0), heads = qt->size(1);
        const double scale = PyFloat_AsDouble(a[8]);
        const long window = PyLong_AsLong(a[9]);
        if (PyErr_Occurred()) return nullptr;
        const int want = PyObject_IsTrue(a[11]);
        if (want < 0) return nullptr;
        if (window > INT32_MAX || window < INT32_MIN) return refuse("window=%ld", window);
        Rows q, out;
        Table t;
        const int32_t* lengths;
        if (!few_enough(rows) || !few_enough(heads) || !rows_operand("q", a[5], c, rows, heads, q) || !table_operand(a[6], c, t) ||
            !index_operand("lengths", a[7], c, rows, lengths))
            return nullptr;
        if (t.rows != rows) return refuse("table must have q's %lld rows", (long long)rows);
        // the workspace first: without one the caller has to make it and call again
        void* ws = nullptr;
        size_t ws_bytes = 0;
        const size_t need = exq_attend_workspace_bytes(c.cache, (int)rows, (int)heads, t.width);
        if (need) {
            const at::Tensor* w = nullptr;
            if (a[13] != Py_None) {
                if (!(w = tensor("workspace", a[13]))) return nullptr;
                if (!w->is_cuda() || w->get_device() != c.index || !w->is_contiguous())
                    return refuse("workspace must be contiguous on cuda:%d", c.index);
            } else if (a[14] != Py_None) {
                if (!(w = tensor("workspace", a[14]))) return nullptr;
                if (w->nbytes() < need) w = nullptr;
            }
            if (!w) return PyLong_FromSize_t(need);
            ws = w->data_ptr();
            ws_bytes = w->nbytes();
        }
        THPObjectPtr out_o(a[10] == Py_None ? THPVariable_Wrap(empty(c, {rows, heads, c.dim}, at::kHalf)) : Py_NewRef(a[10]));
        if (!out_o || !rows_operand("out", out_o, c, rows, heads, out)) return nullptr;
        THPObjectPtr lse_o;
        float* lse = nullptr;
        if (a[12] != Py_None || want) {
            lse_o = a[12] == Py_None ? THPVariable_Wrap(empty(c, {rows, heads}, at::kFloat)) : Py_NewRef(a[12]);
            const at::Tensor* l = lse_o ? tensor("lse", lse_o) : nullptr;
            if (!l) return nullptr;
            if (!(here(*l, c, at::kFloat) && l->dim() == 2 && l->size(0) == rows && l->size(1) == heads && l->is_contiguous()))
                return refuse("lse must be contiguous fp32 [%lld][%lld] on cuda:%d", (long long)rows, (long long)heads, c.index);
            lse = static_cast<float*>(l->data_ptr());
        }
        THPObjectPtr value(want ? PyTuple_Pack(2, out_o.get(), lse_o.get()) : Py_NewRef(out_o.get()));
        if (!value) return nullptr;
        const exq_status st = exq_attend(c.cache, q.p, q.row, q.head, (int)rows, (int)heads, t.p, t.width, t.stride, lengths,
                                         (float)scale, (int)window, out.p, out.row, out.head, lse, ws, ws_bytes, c.stream);
        return status_or(st, "exq_attend", std::move(value));
    });
}

PyObject* set_error(PyObject*, PyObject* cls) {
    Py_XDECREF(g_error);
    g_error = Py_NewRef(cls);
    Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(read)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_exq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__exq_torch() { return PyModule_Create(&module); }
