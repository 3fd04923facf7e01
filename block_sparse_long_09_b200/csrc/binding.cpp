// binding.cpp -- tensor checks and calls of the paged-cache entry points for the Python binding.
//
// A decode step's calls take 2 to 10 us on the GPU; checking a dozen tensors and passing
// them on from Python took 20 us.  This module reads dtype, shape, strides and device of
// the tensors directly, allocates outputs and workspace with torch's allocator, and calls the
// C ABI through the addresses that qsa.py takes from the library it has loaded.  Wrong arguments raise
// ValueError before any CUDA call; the functions return the C ABI's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "qsa.h"

namespace {

struct Api {
    decltype(&qsa_cache_write_paged) write = nullptr;
    decltype(&qsa_cache_read_paged) read = nullptr;
    decltype(&qsa_chunk_attn_paged) chunk = nullptr;
    decltype(&qsa_rope_axes) rope = nullptr;
    decltype(&qsa_workspace_size) workspace = nullptr;
} api;

constexpr int64_t kHQ = 24, kHKV = 2, kD = 256;

std::string shape_of(const at::Tensor &t)
{
    std::string s = std::string(c10::toString(t.scalar_type())) + " (";
    for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.is_contiguous() ? ")" : "), strided");
}

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

// a tensor argument; undefined for None
at::Tensor tensor(PyObject *o, const char *name, bool optional = false)
{
    if (o == Py_None) {
        if (!optional) refuse(std::string(name) + " is needed");
        return at::Tensor();
    }
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

// packed rows: bf16 [rows, heads, 256], contiguous (the kernels cannot see the extent)
void check_rows(const at::Tensor &t, const char *name, int64_t heads, int64_t rows = -1)
{
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(1) != heads || t.size(2) != kD ||
        !t.is_contiguous() || (rows >= 0 && t.size(0) != rows))
        refuse(std::string(name) + " must be contiguous bf16 [" + (rows >= 0 ? std::to_string(rows) : "rows") + ", " +
               std::to_string(heads) + ", 256], got " + shape_of(t));
}

// int32, contiguous, of the given extents (-1: any)
void check_i32(const at::Tensor &t, const char *name, std::initializer_list<int64_t> shape)
{
    bool ok = t.scalar_type() == at::kInt && t.dim() == (int64_t)shape.size() && t.is_contiguous();
    int64_t i = 0;
    for (int64_t want : shape) {
        ok = ok && (want < 0 || t.size(i) == want);
        ++i;
    }
    if (!ok) refuse(std::string(name) + " must be contiguous int32 of the call's shape, got " + shape_of(t));
}

struct Pool {
    at::Tensor k, v, ks, vs, table;
    int32_t format;
    int64_t pages;
    int32_t page_size, cols;
};

Pool pool(PyObject *const *k_v_table_ks_vs, int64_t batch)
{
    PyObject *const *a = k_v_table_ks_vs;
    Pool p;
    p.k = tensor(a[0], "k_pages");
    p.v = tensor(a[1], "v_pages");
    p.table = tensor(a[2], "block_table");
    p.ks = tensor(a[3], "k_scales", true);
    p.vs = tensor(a[4], "v_scales", true);
    const auto type = p.k.scalar_type();
    if ((type != at::kBFloat16 && type != at::kFloat8_e4m3fn) || p.v.scalar_type() != type)
        refuse("pages must be bfloat16 or float8_e4m3fn, both alike, got " + shape_of(p.k) + " and " + shape_of(p.v));
    if (p.k.dim() != 4 || p.k.size(2) != kHKV || p.k.size(3) != kD || p.k.sizes() != p.v.sizes() ||
        !p.k.is_contiguous() || !p.v.is_contiguous())
        refuse("pages must be contiguous [num_pages, page_size, 2, 256], got " + shape_of(p.k) + " and " + shape_of(p.v));
    check_i32(p.table, "block_table", {batch, -1});
    p.format = type == at::kBFloat16 ? QSA_CACHE_BF16 : QSA_CACHE_E4M3;
    p.pages = p.k.size(0);
    if (p.k.size(1) > INT32_MAX || p.table.size(1) > INT32_MAX) refuse("pages or block_table too large");
    p.page_size = (int32_t)p.k.size(1);
    p.cols = (int32_t)p.table.size(1);
    if (p.format == QSA_CACHE_E4M3) {
        for (const at::Tensor *t : {&p.ks, &p.vs})
            if (!t->defined() || t->scalar_type() != at::kByte || t->dim() != 3 ||
                t->sizes() != p.k.sizes().slice(0, 3) || !t->is_contiguous())
                refuse("k_scales and v_scales must be contiguous uint8 [num_pages, page_size, 2] for float8_e4m3fn pages");
    } else if (p.ks.defined() || p.vs.defined()) {
        refuse("bfloat16 pages have no scales");
    }
    return p;
}

// sequences of a prefix-sum argument
int64_t batch_of(const at::Tensor &cu, const char *name)
{
    if (cu.scalar_type() != at::kInt || cu.dim() != 1 || !cu.is_contiguous() || cu.size(0) < 2)
        refuse(std::string(name) + " must be contiguous int32 [batch + 1], got " + shape_of(cu));
    return cu.size(0) - 1;
}

// every tensor on one CUDA device, the current one: calls launch on its current stream
void check_device(const at::Tensor &first, std::initializer_list<const at::Tensor *> rest)
{
    if (!first.is_cuda()) refuse("tensors must be on a CUDA device");
    for (const at::Tensor *t : rest)
        if (t->defined() && t->device() != first.device())
            refuse("tensors on " + first.device().str() + " and " + t->device().str() + " in one call");
    if (first.device().index() != c10::cuda::current_device())
        refuse("tensors on " + first.device().str() + ", but the current device is cuda:" +
               std::to_string((int)c10::cuda::current_device()));
}

void *stream_of(const at::Tensor &t) { return c10::cuda::getCurrentCUDAStream(t.device().index()).stream(); }

template <typename T>
T *ptr(const at::Tensor &t) { return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr; }

int64_t integer(PyObject *o, const char *name, int64_t lo, int64_t hi)
{
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) {
        PyErr_Clear();
        refuse(std::string(name) + " must be an integer");
    }
    if (x < lo || x > hi) refuse(std::string(name) + " = " + std::to_string(x) + " is out of range");
    return x;
}

const qsa_config *config(PyObject *o) { return static_cast<const qsa_config *>(PyLong_AsVoidPtr(o)); }

at::Tensor empty(at::IntArrayRef size, at::ScalarType type, const at::Tensor &like)
{
    return at::detail::empty_cuda(size, type, like.device(), std::nullopt);
}

// every function's frame: the argument count, and C++ exceptions as Python ones
template <typename F>
PyObject *guarded(Py_ssize_t n, Py_ssize_t want, F f)
{
    if (n != want || api.write == nullptr) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or the library is not bound");
        return nullptr;
    }
    try {
        return f();
    } catch (const std::invalid_argument &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch != nullptr ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        PyErr_SetString(type != nullptr ? type : PyExc_MemoryError, e.what());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (cfg, k, v, k_pages, v_pages, block_table, k_scales, v_scales, cu_q, cu_k) -> status
PyObject *cache_write_paged(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor k = tensor(a[1], "k"), v = tensor(a[2], "v"), cu_q = tensor(a[8], "cu_seqlens_q"),
                         cu_k = tensor(a[9], "cu_seqlens_k");
        const int64_t batch = batch_of(cu_q, "cu_seqlens_q");
        const Pool p = pool(a + 3, batch);
        check_rows(k, "k", kHKV);
        check_rows(v, "v", kHKV, k.size(0));
        check_i32(cu_k, "cu_seqlens_k", {batch + 1});
        check_device(k, {&v, &p.k, &p.v, &p.ks, &p.vs, &p.table, &cu_q, &cu_k});
        return PyLong_FromLong(api.write(config(a[0]), ptr<qsa_bf16>(k), ptr<qsa_bf16>(v), ptr<int32_t>(cu_q),
                                         ptr<int32_t>(cu_k), (int32_t)batch, k.size(0), p.format, ptr<void>(p.k),
                                         ptr<void>(p.v), ptr<uint8_t>(p.ks), ptr<uint8_t>(p.vs), p.pages, p.page_size,
                                         ptr<int32_t>(p.table), p.cols, stream_of(k)));
    });
}

// (cfg, k_pages, v_pages, block_table, k_scales, v_scales, cu_k, cu_out, total_out, tok_begin, k, v)
// -> (status, k, v)
PyObject *cache_read_paged(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 12, [&]() -> PyObject * {
        const at::Tensor cu_k = tensor(a[6], "cu_seqlens_k"), cu_out = tensor(a[7], "cu_out"),
                         begin = tensor(a[9], "tok_begin", true);
        at::Tensor k = tensor(a[10], "k", true), v = tensor(a[11], "v", true);
        const int64_t batch = batch_of(cu_k, "cu_seqlens_k"), total = integer(a[8], "total_out", 0, INT32_MAX);
        const Pool p = pool(a + 1, batch);
        check_i32(cu_out, "cu_out", {batch + 1});
        if (begin.defined()) check_i32(begin, "tok_begin", {batch});
        if (k.defined()) check_rows(k, "k", kHKV, total);
        if (v.defined()) check_rows(v, "v", kHKV, total);
        check_device(p.k, {&p.v, &p.ks, &p.vs, &p.table, &cu_k, &cu_out, &begin, &k, &v});
        if (!k.defined()) k = empty({total, kHKV, kD}, at::kBFloat16, p.k);
        if (!v.defined()) v = empty({total, kHKV, kD}, at::kBFloat16, p.k);
        const long st = api.read(config(a[0]), p.format, ptr<void>(p.k), ptr<void>(p.v), ptr<uint8_t>(p.ks),
                                 ptr<uint8_t>(p.vs), p.pages, p.page_size, ptr<int32_t>(p.table), p.cols,
                                 ptr<int32_t>(cu_k), ptr<int32_t>(begin), ptr<int32_t>(cu_out), (int32_t)batch, total,
                                 ptr<qsa_bf16>(k), ptr<qsa_bf16>(v), stream_of(p.k));
        return Py_BuildValue("(lNN)", st, THPVariable_Wrap(k), THPVariable_Wrap(v));
    });
}

// (cfg, q, k_pages, v_pages, block_table, k_scales, v_scales, cu_q, cu_k, max_len_q, max_len_k, window, sinks, o,
//  lse, want_lse, ws) -> (status, o, lse)
PyObject *chunk_attn_paged(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 17, [&]() -> PyObject * {
        const at::Tensor q = tensor(a[1], "q"), cu_q = tensor(a[7], "cu_seqlens_q"), cu_k = tensor(a[8], "cu_seqlens_k");
        at::Tensor o = tensor(a[13], "o", true), lse = tensor(a[14], "lse", true), ws = tensor(a[16], "ws", true);
        const int64_t batch = batch_of(cu_q, "cu_seqlens_q");
        const Pool p = pool(a + 2, batch);
        const int32_t max_q = (int32_t)integer(a[9], "max_len_q", 0, INT32_MAX);
        const int64_t max_k = integer(a[10], "max_len_k", 0, INT32_MAX);
        const int32_t window = (int32_t)integer(a[11], "window", 0, INT32_MAX);
        const int32_t sinks = (int32_t)integer(a[12], "sinks", 0, INT32_MAX);
        check_rows(q, "q", kHQ);
        check_i32(cu_k, "cu_seqlens_k", {batch + 1});
        if (o.defined()) check_rows(o, "o", kHQ, q.size(0));
        if (lse.defined() && (lse.scalar_type() != at::kFloat || lse.dim() != 2 || lse.size(0) != q.size(0) ||
                              lse.size(1) != kHQ || !lse.is_contiguous()))
            refuse("lse must be contiguous fp32 [" + std::to_string(q.size(0)) + ", 24], got " + shape_of(lse));
        if (ws.defined() && (ws.scalar_type() != at::kByte || !ws.is_contiguous()))
            refuse("ws must be contiguous uint8, got " + shape_of(ws));
        check_device(q, {&p.k, &p.v, &p.ks, &p.vs, &p.table, &cu_q, &cu_k, &o, &lse, &ws});
        const qsa_config *cfg = config(a[0]);
        if (!o.defined()) o = empty(q.sizes(), at::kBFloat16, q);
        if (!lse.defined() && PyObject_IsTrue(a[15]) == 1) lse = empty({q.size(0), kHQ}, at::kFloat, q);
        if (!ws.defined())
            ws = empty({(int64_t)api.workspace(cfg, QSA_OP_CHUNK_PAGED, (int32_t)batch, q.size(0), max_k)}, at::kByte, q);
        const long st = api.chunk(cfg, ptr<qsa_bf16>(q), p.format, ptr<void>(p.k), ptr<void>(p.v), ptr<uint8_t>(p.ks),
                                  ptr<uint8_t>(p.vs), p.pages, p.page_size, ptr<int32_t>(p.table), p.cols,
                                  ptr<int32_t>(cu_q), ptr<int32_t>(cu_k), (int32_t)batch, q.size(0), max_q, window,
                                  sinks, ptr<qsa_bf16>(o), ptr<float>(lse), ptr<void>(ws), (size_t)ws.numel(),
                                  stream_of(q));
        PyObject *l = Py_None;
        if (lse.defined()) l = THPVariable_Wrap(lse);
        else Py_INCREF(l);
        return Py_BuildValue("(lNN)", st, THPVariable_Wrap(o), l);
    });
}

// (cfg, q, k, positions, s0, s1, s2, flags, q_out, k_out) -> (status, q_out, k_out)
PyObject *rope_axes(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded(n, 10, [&]() -> PyObject * {
        const at::Tensor q = tensor(a[1], "q", true), k = tensor(a[2], "k", true), pos = tensor(a[3], "positions");
        at::Tensor qo = tensor(a[8], "q_out", true), ko = tensor(a[9], "k_out", true);
        if (!q.defined() && !k.defined()) refuse("q or k is needed");
        const at::Tensor &x = q.defined() ? q : k;
        if (x.dim() != 3) refuse("q and k must be [rows, heads, 256], got " + shape_of(x));
        const int64_t total = x.size(0);
        check_i32(pos, "positions", {3, total});
        if (q.defined()) check_rows(q, "q", kHQ, total);
        if (k.defined()) check_rows(k, "k", kHKV, total);
        if ((qo.defined() && !q.defined()) || (ko.defined() && !k.defined())) refuse("an output without its input");
        if (qo.defined()) check_rows(qo, "q_out", kHQ, total);
        if (ko.defined()) check_rows(ko, "k_out", kHKV, total);
        int32_t s[3];
        for (int i = 0; i < 3; ++i) s[i] = (int32_t)integer(a[4 + i], "a section", INT32_MIN, INT32_MAX);
        const uint32_t flags = (uint32_t)integer(a[7], "flags", 0, UINT32_MAX);
        check_device(x, {&q, &k, &pos, &qo, &ko});
        if (q.defined() && !qo.defined()) qo = empty(q.sizes(), at::kBFloat16, q);
        if (k.defined() && !ko.defined()) ko = empty(k.sizes(), at::kBFloat16, k);
        const long st = api.rope(config(a[0]), ptr<qsa_bf16>(q), ptr<qsa_bf16>(k), ptr<int32_t>(pos), total, s[0], s[1],
                                 s[2], flags, ptr<qsa_bf16>(qo), ptr<qsa_bf16>(ko), stream_of(x));
        PyObject *r[2];
        const at::Tensor *out[2] = {&qo, &ko};
        for (int i = 0; i < 2; ++i) {
            r[i] = Py_None;
            if (out[i]->defined()) r[i] = THPVariable_Wrap(*out[i]);
            else Py_INCREF(r[i]);
        }
        return Py_BuildValue("(lNN)", st, r[0], r[1]);
    });
}

// (addresses of write, read, chunk, rope, workspace_size)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "five addresses");
        return nullptr;
    }
    api.write = reinterpret_cast<decltype(api.write)>(PyLong_AsVoidPtr(a[0]));
    api.read = reinterpret_cast<decltype(api.read)>(PyLong_AsVoidPtr(a[1]));
    api.chunk = reinterpret_cast<decltype(api.chunk)>(PyLong_AsVoidPtr(a[2]));
    api.rope = reinterpret_cast<decltype(api.rope)>(PyLong_AsVoidPtr(a[3]));
    api.workspace = reinterpret_cast<decltype(api.workspace)>(PyLong_AsVoidPtr(a[4]));
    if (PyErr_Occurred()) return nullptr;
    Py_RETURN_NONE;
}

#define QSA_METHOD(f, doc) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL, doc}
PyMethodDef methods[] = {
    QSA_METHOD(bind, "the library's entry points"),
    QSA_METHOD(cache_write_paged, "qsa_cache_write_paged"),
    QSA_METHOD(cache_read_paged, "qsa_cache_read_paged"),
    QSA_METHOD(chunk_attn_paged, "qsa_chunk_attn_paged"),
    QSA_METHOD(rope_axes, "qsa_rope_axes"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "tensor checks and calls of the paged-cache entry points", -1,
                      methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
