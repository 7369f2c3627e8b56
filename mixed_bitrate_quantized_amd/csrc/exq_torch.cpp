// The calls on PyTorch tensors (the module _exq_torch) of KVCache, PagePool,
// Rotary, Adapters and sample: checks of shapes, types, strides and devices, outputs where none are given, and the call of
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

// Device and stream, which the calls without a cache start with.
Call call_on(PyObject* const* a) {
    Call c{};
    c.index = (int)PyLong_AsLong(a[0]);
    c.stream = PyLong_AsVoidPtr(a[1]);
    return c;
}

// A given output, or a new one.
PyObject* given_or_empty(PyObject* o, const Call& c, at::IntArrayRef shape, at::ScalarType type) {
    return o == Py_None ? THPVariable_Wrap(empty(c, shape, type)) : Py_NewRef(o);
}

// New outputs of a call, contiguous, in one allocation, like the chunks of a tensor: an
// allocation costs the host 1.8 us, a tensor on it a tenth of that.
struct Output {
    at::IntArrayRef shape;
    at::ScalarType type;
    size_t bytes() const {
        int64_t n = (int64_t)at::elementSize(type);
        for (const int64_t x : shape) n *= x;
        return ((size_t)n + 255) / 256 * 256;
    }
};
template <size_t N> void empties(const Call& c, const Output (&x)[N], THPObjectPtr (&out)[N]) {
    size_t total = 0;
    for (const Output& o : x) total += o.bytes();
    const at::Tensor all = empty(c, {(int64_t)total}, at::kByte);
    size_t at = 0;
    for (size_t i = 0; i < N; ++i) {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                                                c10::scalarTypeToTypeMeta(x[i].type));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(x[i].shape);
        t.unsafeGetTensorImpl()->set_storage_offset((int64_t)(at / at::elementSize(x[i].type)));
        at += x[i].bytes();
        out[i] = THPVariable_Wrap(t);
    }
}

// A pool's own arrays.
struct Pool {
    Table t;
    int32_t *lengths, *free_pages, *free_count, *workspace;
    int64_t n_pages, workspace_bytes;
};
bool pool_operand(PyObject* table, PyObject* lengths, PyObject* free, PyObject* count, PyObject* workspace, const Call& c, Pool& p) {
    const at::Tensor *f = tensor("free", free), *w = f ? tensor("workspace", workspace) : nullptr;
    if (!w) return false;
    p.n_pages = f->numel();
    p.workspace_bytes = 4 * w->numel();
    if (!few_enough(p.n_pages) || !table_operand(table, c, p.t)) return false;
    const int32_t *x[4];
    if (!index_operand("lengths", lengths, c, p.t.rows, x[0]) || !index_operand("free", free, c, p.n_pages, x[1]) ||
        !index_operand("free_count", count, c, 1, x[2]) || !index_operand("workspace", workspace, c, w->numel(), x[3]))
        return false;
    p.lengths = const_cast<int32_t*>(x[0]);
    p.free_pages = const_cast<int32_t*>(x[1]);
    p.free_count = const_cast<int32_t*>(x[2]);
    p.workspace = const_cast<int32_t*>(x[3]);
    return true;
}

// extend(device, stream, page_size, table, lengths, free, free_count, served, workspace, counts, rows, seqs or None,
//        positions or None, offsets or None) -> (seqs, positions, offsets)
PyObject* extend(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!arity(n, 14)) return nullptr;
        const Call c = call_on(a);
        const long page_size = PyLong_AsLong(a[2]);
        const long long rows = PyLong_AsLongLong(a[10]);
        if (PyErr_Occurred()) return nullptr;
        if (rows < 0) return refuse("%lld rows", rows);
        Pool p;
        const int32_t *served, *counts, *out[3];
        if (!few_enough(rows) || !pool_operand(a[3], a[4], a[5], a[6], a[8], c, p) || !index_operand("served", a[7], c, 1, served) ||
            !index_operand("counts", a[9], c, p.t.rows, counts))
            return nullptr;
        const char* names[3] = {"seqs", "positions", "offsets"};
        THPObjectPtr o[3];
        const int64_t sizes[3] = {rows, rows, (int64_t)p.t.rows + 1};
        if (a[11] == Py_None && a[12] == Py_None && a[13] == Py_None)
            empties(c, {Output{sizes[0], at::kInt}, Output{sizes[1], at::kInt}, Output{sizes[2], at::kInt}}, o);
        for (int i = 0; i < 3; ++i) {
            const int64_t size = sizes[i];
            if (!o[i]) o[i] = given_or_empty(a[11 + i], c, {size}, at::kInt);
            if (!o[i] || !index_operand(names[i], o[i], c, size, out[i])) return nullptr;
        }
        THPObjectPtr outs(PyTuple_Pack(3, o[0].get(), o[1].get(), o[2].get()));
        if (!outs) return nullptr;
        return status_or(exq_pages_extend(const_cast<int32_t*>(p.t.p), p.t.rows, p.t.width, p.t.stride, (int)page_size, p.lengths,
                                          counts, p.free_pages, p.free_count, (int)p.n_pages, const_cast<int32_t*>(out[0]),
                                          const_cast<int32_t*>(out[1]), (int)rows, const_cast<int32_t*>(out[2]),
                                          const_cast<int32_t*>(served), p.workspace, p.workspace_bytes, c.stream),
                         "exq_pages_extend", std::move(outs));
    });
}

// trim(device, stream, page_size, table, lengths, free, free_count, workspace, keep)
PyObject* trim(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!arity(n, 9)) return nullptr;
        const Call c = call_on(a);
        const long page_size = PyLong_AsLong(a[2]);
        if (PyErr_Occurred()) return nullptr;
        Pool p;
        const int32_t* keep;
        if (!pool_operand(a[3], a[4], a[5], a[6], a[7], c, p) || !index_operand("keep", a[8], c, p.t.rows, keep)) return nullptr;
        return status_or(exq_pages_trim(const_cast<int32_t*>(p.t.p), p.t.rows, p.t.width, p.t.stride, (int)page_size, p.lengths, keep,
                                        p.free_pages, p.free_count, (int)p.n_pages, p.workspace, p.workspace_bytes, c.stream),
                         "exq_pages_trim", THPObjectPtr(Py_NewRef(Py_None)));
    });
}

// rotate(device, stream, head_dim, rotary_dim, interleaved, rates, factor, q, positions, k or None, q_out or None,
//        k_out or None) -> q_out, or (q_out, k_out)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!arity(n, 12)) return nullptr;
        Call c = call_on(a);
        c.dim = PyLong_AsLongLong(a[2]);
        const long part = PyLong_AsLong(a[3]);
        const int interleaved = PyObject_IsTrue(a[4]);
        const double factor = PyFloat_AsDouble(a[6]);
        if (PyErr_Occurred()) return nullptr;
        const at::Tensor *rates = tensor("rates", a[5]), *qt = rates ? tensor("q", a[7]) : nullptr;
        if (!qt) return nullptr;
        if (!here(*rates, c, at::kDouble) || rates->dim() != 1 || !rates->is_contiguous() || 2 * rates->size(0) != part)
            return refuse("rates must be contiguous fp64 [%ld] on cuda:%d", part / 2, c.index);
        if (qt->dim() != 3) return refuse("q must be [rows][heads][head_dim]");
        const int64_t rows = qt->size(0);
        const bool both = a[9] != Py_None;
        if (!both && a[11] != Py_None) return refuse("k_out without k");
        int64_t heads[2] = {qt->size(1), 0};
        if (both) {
            const at::Tensor* kt = tensor("k", a[9]);
            if (!kt) return nullptr;
            if (kt->dim() != 3) return refuse("k must be [rows][heads][head_dim]");
            heads[1] = kt->size(1);
        }
        const int32_t* positions;
        Rows in[2] = {}, out[2] = {};
        THPObjectPtr o[2];
        if (!few_enough(rows) || !few_enough(heads[0]) || !few_enough(heads[1]) || !index_operand("positions", a[8], c, rows, positions))
            return nullptr;
        for (int i = 0; i < (both ? 2 : 1); ++i)
            if (!rows_operand(i ? "k" : "q", a[i ? 9 : 7], c, rows, heads[i], in[i])) return nullptr;
        if (both && a[10] == Py_None && a[11] == Py_None) {
            const int64_t q_shape[3] = {rows, heads[0], c.dim}, k_shape[3] = {rows, heads[1], c.dim};
            empties(c, {Output{q_shape, at::kHalf}, Output{k_shape, at::kHalf}}, o);
        }
        for (int i = 0; i < (both ? 2 : 1); ++i) {
            if (!o[i]) o[i] = given_or_empty(a[10 + i], c, {rows, heads[i], c.dim}, at::kHalf);
            if (!o[i] || !rows_operand(i ? "k_out" : "q_out", o[i], c, rows, heads[i], out[i])) return nullptr;
        }
        THPObjectPtr value(both ? PyTuple_Pack(2, o[0].get(), o[1].get()) : Py_NewRef(o[0].get()));
        if (!value) return nullptr;
        return status_or(exq_rotate(in[0].p, in[0].row, in[0].head, out[0].p, out[0].row, out[0].head, (int)heads[0], in[1].p,
                                    in[1].row, in[1].head, out[1].p, out[1].row, out[1].head, (int)heads[1], (int)rows, (int)c.dim,
                                    (int)part, interleaved, static_cast<const double*>(rates->data_ptr()), (float)factor, positions,
                                    c.stream),
                         "exq_rotate", std::move(value));
    });
}

// An fp16 matrix [rows][width] with contiguous rows.
bool matrix_operand(const char* name, PyObject* o, const Call& c, int64_t rows, int64_t width, Rows& r) {
    const at::Tensor* t = tensor(name, o);
    if (!t) return false;
    if (!here(*t, c, at::kHalf) || t->dim() != 2 || t->size(0) != rows || t->size(1) != width || t->stride(1) != 1) {
        refuse("%s must be fp16 [%lld][%lld] on cuda:%d with contiguous rows", name, (long long)rows, (long long)width, c.index);
        return false;
    }
    r = Rows{t->data_ptr(), rows > 1 ? t->stride(0) : 0, 0};
    return true;
}

// lora_add(device, stream, adapters, K, N, x, ids, y, out or None, workspace or None) -> out
PyObject* lora_add(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!arity(n, 10)) return nullptr;
        const Call c = call_on(a);
        const exq_adapters_t h = a[2] == Py_None ? nullptr : static_cast<exq_adapters_t>(PyLong_AsVoidPtr(a[2]));
        const int64_t K = PyLong_AsLongLong(a[3]), N = PyLong_AsLongLong(a[4]);
        if (PyErr_Occurred()) return nullptr;
        const at::Tensor* xt = tensor("x", a[5]);
        if (!xt) return nullptr;
        if (xt->dim() != 2) return refuse("x must be [rows][K]");
        const int64_t rows = xt->size(0);
        Rows x, y, out;
        const int32_t* ids;
        if (!few_enough(rows) || !matrix_operand("x", a[5], c, rows, K, x) || !index_operand("ids", a[6], c, rows, ids) ||
            !matrix_operand("y", a[7], c, rows, N, y))
            return nullptr;
        THPObjectPtr out_o(given_or_empty(a[8], c, {rows, N}, at::kHalf));
        if (!out_o || !matrix_operand("out", out_o, c, rows, N, out)) return nullptr;
        const size_t need = exq_lora_workspace_bytes(h, (int)rows);
        at::Tensor own;
        const at::Tensor* w = nullptr;
        if (a[9] != Py_None) {
            if (!(w = tensor("workspace", a[9]))) return nullptr;
            if (!w->is_cuda() || w->get_device() != c.index || !w->is_contiguous())
                return refuse("workspace must be contiguous on cuda:%d", c.index);
        } else if (need) {
            own = empty(c, {(int64_t)need}, at::kByte);
            w = &own;
        }
        return status_or(exq_lora_add(h, x.p, x.row, (int)rows, ids, y.p, y.row, out.p, out.row, w ? w->data_ptr() : nullptr,
                                      w ? w->nbytes() : 0, c.stream),
                         "exq_lora_add", std::move(out_o));
    });
}

// A setting of every row: a tensor of them, or a number for all.
template <class T> struct Setting {
    const T* p = nullptr;
    T all = 0;
};
bool setting(const char* name, PyObject* o, const Call& c, int64_t rows, Setting<float>& s) {
    if (!THPVariable_Check(o)) {
        s.all = (float)PyFloat_AsDouble(o);
        return !PyErr_Occurred();
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!here(t, c, at::kFloat) || t.dim() != 1 || t.size(0) != rows || (rows > 1 && t.stride(0) != 1)) {
        refuse("%s must be a number or contiguous fp32 [%lld] on cuda:%d", name, (long long)rows, c.index);
        return false;
    }
    s.p = static_cast<const float*>(t.data_ptr());
    return true;
}
bool setting(const char* name, PyObject* o, const Call& c, int64_t rows, Setting<int32_t>& s) {
    if (THPVariable_Check(o)) return index_operand(name, o, c, rows, s.p);
    const long long x = PyLong_AsLongLong(o);
    if (PyErr_Occurred()) return false;
    s.all = x > INT32_MAX ? INT32_MAX : x < 0 ? 0 : (int32_t)x;
    return true;
}

// sample(device, stream, logits, u, temperature, top_k, top_p, min_p, out or None, return_logprobs, logprobs or None)
//   -> tokens, or (tokens, logprobs)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded([&]() -> PyObject* {
        if (!arity(n, 11)) return nullptr;
        const Call c = call_on(a);
        const int want = PyObject_IsTrue(a[9]);
        if (PyErr_Occurred()) return nullptr;
        const at::Tensor* l = tensor("logits", a[2]);
        if (!l) return nullptr;
        const bool wide = l->scalar_type() == at::kFloat;
        if (!here(*l, c, wide ? at::kFloat : at::kHalf) || l->dim() != 2 || (l->size(1) > 1 && l->stride(1) != 1))
            return refuse("logits must be fp16 or fp32 [rows][vocab] on cuda:%d with contiguous rows", c.index);
        const int64_t rows = l->size(0), vocab = l->size(1);
        Setting<float> u, temperature, top_p, min_p;
        Setting<int32_t> top_k;
        if (!few_enough(rows) || !few_enough(vocab)) return nullptr;
        if (!THPVariable_Check(a[3])) return refuse("u must be a tensor");
        if (!setting("u", a[3], c, rows, u) || !setting("temperature", a[4], c, rows, temperature) ||
            !setting("top_k", a[5], c, rows, top_k) || !setting("top_p", a[6], c, rows, top_p) ||
            !setting("min_p", a[7], c, rows, min_p))
            return nullptr;
        THPObjectPtr tokens, logs;
        if (want && a[8] == Py_None && a[10] == Py_None) {
            THPObjectPtr o[2];
            empties(c, {Output{rows, at::kInt}, Output{rows, at::kFloat}}, o);
            tokens = std::move(o[0]);
            logs = std::move(o[1]);
        } else {
            tokens = given_or_empty(a[8], c, {rows}, at::kInt);
        }
        const int32_t* tokens_p;
        if (!tokens || !index_operand("out", tokens, c, rows, tokens_p)) return nullptr;
        float* logs_p = nullptr;
        if (want || a[10] != Py_None) {
            if (!logs) logs = given_or_empty(a[10], c, {rows}, at::kFloat);
            const at::Tensor* t = logs ? tensor("logprobs", logs) : nullptr;
            if (!t) return nullptr;
            if (!here(*t, c, at::kFloat) || t->dim() != 1 || t->size(0) != rows || (rows > 1 && t->stride(0) != 1))
                return refuse("logprobs must be contiguous fp32 [%lld] on cuda:%d", (long long)rows, c.index);
            logs_p = static_cast<float*>(t->data_ptr());
        }
        THPObjectPtr value(want ? PyTuple_Pack(2, tokens.get(), logs.get()) : Py_NewRef(tokens.get()));
        if (!value) return nullptr;
        const size_t bytes = exq_sample_workspace_bytes((int)rows, (int)vocab);
        at::Tensor workspace;
        if (bytes) workspace = empty(c, {(int64_t)bytes}, at::kByte);
        return status_or(exq_sample(l->data_ptr(), wide ? 32 : 16, (int)rows, (int)vocab, rows > 1 ? l->stride(0) : 0, u.p,
                                    temperature.p, temperature.all, top_k.p, top_k.all, top_p.p, top_p.all, min_p.p, min_p.all,
                                    const_cast<int32_t*>(tokens_p), logs_p, bytes ? workspace.data_ptr() : nullptr, bytes, c.stream),
                         "exq_sample", std::move(value));
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
    {"extend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(extend)), METH_FASTCALL, nullptr},
    {"trim", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(trim)), METH_FASTCALL, nullptr},
    {"rotate", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rotate)), METH_FASTCALL, nullptr},
    {"lora_add", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(lora_add)), METH_FASTCALL, nullptr},
    {"sample", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(sample)), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_exq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__exq_torch() { return PyModule_Create(&module); }
