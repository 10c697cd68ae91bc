// marshal.cpp -- argument structures of include/pq2_attention.h from torch
// tensors, for the Python binding (gemm_int8_act_amd/attention.py).
//
// The attention calls of a decode step take up to eleven tensors; reading and
// checking their attributes from Python costs 5 to 10 us a call, more than the
// kernels run.  Here it is under 1 us.  Each function checks what Python
// callers may get wrong (types, shapes, strides, one device), raises
// ValueError, and returns (the packed structure, the device); nothing is
// launched or kept.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <torch/csrc/autograd/python_variable.h>

#include "../../include/pq2_attention.h"

#include <exception>

namespace {

struct Refused {};  // the Python error is set

template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
    PyErr_Format(PyExc_ValueError, format, a...);
    throw Refused{};
}

struct Call {
    int64_t device = -2;

    // The tensor behind a Python argument, of one device with the others; null for None.
    const at::Tensor* get(PyObject* o, const char* name) {
        if (o == Py_None) return nullptr;
        if (!THPVariable_Check(o)) refuse("%s: a tensor expected", name);
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided) refuse("%s: a dense tensor expected", name);
        return &t;
    }
    const at::Tensor& must(PyObject* o, const char* name) {
        const at::Tensor* t = get(o, name);
        if (!t) refuse("%s: a tensor expected", name);
        return *t;
    }
    void* pointer(const at::Tensor& t) {
        const int64_t d = t.is_cuda() ? t.get_device() : -1;
        if (device == -2) device = d;
        if (d != device) refuse("all tensors of a call must be on one device");
        return t.data_ptr();
    }
};

int dtype(at::ScalarType s, bool half, const char* name) {
    if (s == at::kBFloat16) return PQ2_BF16;
    if (s == at::kHalf) return PQ2_F16;
    if (s == at::kFloat && !half) return PQ2_F32;
    refuse("%s: unsupported dtype (bf16, f16%s expected)", name, half ? "" : " or f32");
}

// A tensor of heads [rows][heads][head_dim]; strides of single rows and heads
// are those of a contiguous tensor, whatever the tensor says.
struct Heads {
    void* p = nullptr;
    int64_t stride = 0, head = 0, rows = 0, heads = 0, dim = 0;
    at::ScalarType type = at::kFloat;
};

Heads heads(Call& c, PyObject* o, const char* name) {
    const at::Tensor& t = c.must(o, name);
    if (t.dim() != 3) refuse("%s must be [rows][heads][head_dim]", name);
    const auto size = t.sizes(), stride = t.strides();
    if (stride[2] != 1 && size[2] > 1) refuse("%s must have unit stride inside a head", name);
    Heads h;
    h.rows = size[0], h.heads = size[1], h.dim = size[2];
    h.head = h.heads == 1 ? h.dim : stride[1];
    h.stride = h.rows == 1 ? h.heads * h.dim : stride[0];
    h.type = t.scalar_type();
    h.p = c.pointer(t);
    return h;
}

Heads heads_like(Call& c, PyObject* o, const char* name, int64_t rows, int64_t n, int64_t dim, at::ScalarType type) {
    const Heads h = heads(c, o, name);
    if (h.rows != rows || h.heads != n || h.dim != dim) refuse("%s: shape mismatch with the call's other tensors", name);
    if (h.type != type) refuse("%s: dtype mismatch with the call's other tensors", name);
    return h;
}

const int32_t* index(Call& c, PyObject* o, const char* name, int64_t n) {
    const at::Tensor& t = c.must(o, name);
    if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
        refuse("%s must be a contiguous int32 tensor of %lld elements", name, (long long)n);
    return static_cast<const int32_t*>(c.pointer(t));
}

int64_t length(Call& c, PyObject* o, const char* name) {
    const at::Tensor& t = c.must(o, name);
    if (t.dim() != 1) refuse("%s must be a contiguous int32 tensor", name);
    return t.size(0);
}

struct Table {
    const int32_t* p;
    int64_t stride, pages;
};

Table table(Call& c, PyObject* o, int64_t seqs) {
    const at::Tensor& t = c.must(o, "table");
    if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != seqs || (t.stride(1) != 1 && t.size(1) > 1))
        refuse("table must be int32 [sequences][pages] with unit column stride");
    return {static_cast<const int32_t*>(c.pointer(t)), seqs > 1 ? t.stride(0) : t.size(1), t.size(1)};
}

struct Cache {
    void* p;
    int64_t pages;
};

// kv < 0: as many heads as the pages have room for, into *kv.
Cache cache(Call& c, PyObject* o, int64_t page_tokens, int64_t* kv, int64_t dim) {
    const at::Tensor& t = c.must(o, "cache");
    if (t.scalar_type() != at::kByte || t.dim() != 2 || !t.is_contiguous()) refuse("cache must be a contiguous uint8 tensor [pages][page bytes]");
    const int64_t one = pq2_kv_page_bytes(page_tokens, 1, dim);
    if (one < 0) refuse("unsupported page_tokens %lld or head_dim %lld", (long long)page_tokens, (long long)dim);
    if (*kv < 0) *kv = t.size(1) / one;
    if (t.size(1) != one * *kv) refuse("cache: pages must have pq2_kv_page_bytes(page_tokens, kv_heads, head_dim) bytes");
    return {c.pointer(t), t.size(0)};
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused{};
    return v;
}

float real(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused{};
    return (float)v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused{};
    return v != 0;
}

template <typename Args>
PyObject* packed(const Call& c, const Args& a) {
    if (c.device < 0) refuse("device tensors expected");
    return Py_BuildValue("(y#L)", reinterpret_cast<const char*>(&a), (Py_ssize_t)sizeof a, (long long)c.device);
}

// k, v, cache, slots, page_tokens, q, q_out, k_out, v_out, cos, sin, positions, interleaved
PyObject* write(PyObject* const* o) {
    Call c;
    pq2_kv_write_args a{};
    const Heads k = heads(c, o[0], "k");
    const Heads v = heads_like(c, o[1], "v", k.rows, k.heads, k.dim, k.type);
    a.k = k.p, a.k_stride = k.stride, a.k_head = k.head;
    a.v = v.p, a.v_stride = v.stride, a.v_head = v.head;
    a.m = k.rows, a.heads = a.kv_heads = k.heads, a.head_dim = k.dim;
    a.in_dtype = a.out_dtype = dtype(k.type, false, "k");
    a.interleaved = truth(o[12]);
    at::ScalarType out = k.type;
    bool any = false;
    auto output = [&](PyObject* t, const char* name, int64_t n) {
        Heads h = heads(c, t, name);
        if (h.rows != k.rows || h.heads != n || h.dim != k.dim) refuse("%s: shape mismatch with the call's other tensors", name);
        if (any && h.type != out) refuse("q_out, k_out and v_out must have one dtype");
        any = true;
        out = h.type;
        a.out_dtype = dtype(out, false, name);
        return h;
    };
    if (o[5] != Py_None) {
        const Heads q = heads(c, o[5], "q");
        if (q.rows != k.rows || q.dim != k.dim || q.type != k.type) refuse("q, k and v must have one dtype, number of rows and head_dim");
        a.q = q.p, a.q_stride = q.stride, a.q_head = q.head, a.heads = q.heads;
    }
    if (o[6] != Py_None) {
        if (!a.q) refuse("q_out goes with q");
        const Heads h = output(o[6], "q_out", a.heads);
        a.q_out = h.p, a.qo_stride = h.stride, a.qo_head = h.head;
    }
    if (o[7] != Py_None) {
        const Heads h = output(o[7], "k_out", k.heads);
        a.k_out = h.p, a.ko_stride = h.stride, a.ko_head = h.head;
    }
    if (o[8] != Py_None) {
        const Heads h = output(o[8], "v_out", k.heads);
        a.v_out = h.p, a.vo_stride = h.stride, a.vo_head = h.head;
    }
    if (o[9] != Py_None || o[10] != Py_None) {
        const at::Tensor &cs = c.must(o[9], "cos"), &sn = c.must(o[10], "sin");
        if (cs.dim() != 2 || cs.sizes() != sn.sizes() || cs.scalar_type() != at::kFloat || sn.scalar_type() != at::kFloat ||
            !cs.is_contiguous() || !sn.is_contiguous())
            refuse("cos and sin must be contiguous float32 [positions][rot_dim / 2] tables");
        a.cos = static_cast<const float*>(c.pointer(cs)), a.sin = static_cast<const float*>(c.pointer(sn));
        a.positions = index(c, o[11], "positions", k.rows);
        a.table_rows = cs.size(0), a.rot_dim = 2 * cs.size(1);
    }
    if (o[2] != Py_None) {
        int64_t kv = k.heads;
        a.page_tokens = integer(o[4]);
        const Cache p = cache(c, o[2], a.page_tokens, &kv, k.dim);
        a.cache = p.p, a.pages = p.pages;
        a.slots = index(c, o[3], "slots", k.rows);
    }
    return packed(c, a);
}

// cache, table, starts, page_tokens, k_out, v_out
PyObject* read(PyObject* const* o) {
    Call c;
    pq2_kv_read_args a{};
    const Heads k = heads(c, o[4], "k_out");
    const Heads v = heads_like(c, o[5], "v_out", k.rows, k.heads, k.dim, k.type);
    a.k_out = k.p, a.ko_stride = k.stride, a.ko_head = k.head;
    a.v_out = v.p, a.vo_stride = v.stride, a.vo_head = v.head;
    a.rows = k.rows, a.kv_heads = k.heads, a.head_dim = k.dim;
    a.out_dtype = dtype(k.type, false, "k_out");
    a.seqs = length(c, o[2], "starts") - 1;
    a.starts = index(c, o[2], "starts", a.seqs + 1);
    const Table t = table(c, o[1], a.seqs);
    a.table = t.p, a.table_stride = t.stride, a.table_pages = t.pages;
    a.page_tokens = integer(o[3]);
    int64_t kv = k.heads;
    const Cache p = cache(c, o[0], a.page_tokens, &kv, k.dim);
    a.cache = p.p, a.pages = p.pages;
    return packed(c, a);
}

// q, cache, table, lens, page_tokens, out, partials, counters, starts, max_new, max_len (None), scale (None), window
PyObject* paged(PyObject* const* o) {
    Call c;
    pq2_attention_paged_args a{};
    const Heads q = heads(c, o[0], "q");
    const Heads out = heads_like(c, o[5], "out", q.rows, q.heads, q.dim, q.type);
    a.q = q.p, a.q_stride = q.stride, a.q_head = q.head;
    a.out = out.p, a.out_stride = out.stride, a.out_head = out.head;
    a.rows = q.rows, a.heads = q.heads, a.head_dim = q.dim;
    a.dtype = dtype(q.type, true, "q");
    a.seqs = length(c, o[3], "lens");
    a.lens = index(c, o[3], "lens", a.seqs);
    const Table t = table(c, o[2], a.seqs);
    a.table = t.p, a.table_stride = t.stride, a.table_pages = t.pages;
    a.page_tokens = integer(o[4]);
    a.kv_heads = -1;
    const Cache p = cache(c, o[1], a.page_tokens, &a.kv_heads, q.dim);
    a.cache = p.p, a.pages = p.pages;
    if (o[8] != Py_None) a.starts = index(c, o[8], "starts", a.seqs + 1);
    else if (a.rows != a.seqs) refuse("without starts, q has one row a sequence");
    a.max_new = integer(o[9]);
    a.max_len = o[10] == Py_None ? t.pages * a.page_tokens : integer(o[10]);
    a.scale = o[11] == Py_None ? 1.0f / sqrtf((float)q.dim) : real(o[11]);
    a.window = integer(o[12]);
    int64_t floats = 0, words = 0;
    if (pq2_attention_paged_workspace(a.seqs, a.max_new, a.heads, a.kv_heads, a.head_dim, a.max_len, &floats, &words) != PQ2_OK)
        refuse("unsupported sizes (sequences, max_new, heads, kv_heads, head_dim or max_len)");
    if (words) {
        const at::Tensor *f = c.get(o[6], "partials"), *w = c.get(o[7], "counters");
        if (!f || !w || f->scalar_type() != at::kFloat || w->scalar_type() != at::kInt || f->numel() < floats ||
            w->numel() < words || !f->is_contiguous() || !w->is_contiguous())
            refuse("partials float32 and counters int32 of pq2_attention_paged_workspace(...) expected");
        a.partials = static_cast<float*>(c.pointer(*f)), a.counters = static_cast<uint32_t*>(c.pointer(*w));
    }
    return packed(c, a);
}

// q, k, v, out, starts_q, starts_k, causal, scale (None), window
PyObject* prompt(PyObject* const* o) {
    Call c;
    pq2_attention_prompt_args a{};
    const Heads q = heads(c, o[0], "q"), k = heads(c, o[1], "k");
    const Heads v = heads_like(c, o[2], "v", k.rows, k.heads, k.dim, q.type);
    const Heads out = heads_like(c, o[3], "out", q.rows, q.heads, q.dim, q.type);
    if (k.dim != q.dim || k.type != q.type) refuse("q, k, v and out must have one dtype and one head_dim");
    a.q = q.p, a.q_stride = q.stride, a.q_head = q.head;
    a.k = k.p, a.k_stride = k.stride, a.k_head = k.head;
    a.v = v.p, a.v_stride = v.stride, a.v_head = v.head;
    a.out = out.p, a.out_stride = out.stride, a.out_head = out.head;
    a.rows_q = q.rows, a.rows_k = k.rows, a.heads = q.heads, a.kv_heads = k.heads, a.head_dim = q.dim;
    a.dtype = dtype(q.type, true, "q");
    a.seqs = length(c, o[4], "starts_q") - 1;
    a.starts_q = index(c, o[4], "starts_q", a.seqs + 1);
    a.starts_k = index(c, o[5], "starts_k", a.seqs + 1);
    a.causal = truth(o[6]);
    a.scale = o[7] == Py_None ? 1.0f / sqrtf((float)q.dim) : real(o[7]);
    a.window = integer(o[8]);
    return packed(c, a);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* o, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
    try {
        return F(o);
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception& e) {
        return PyErr_Format(PyExc_ValueError, "%s", e.what());
    }
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<write, 13>("kv_write"), method<read, 6>("kv_read"), method<paged, 13>("attention_paged"),
                         method<prompt, 9>("attention_prompt"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the torch whose tensors this code reads.
PyMODINIT_FUNC PyInit__marshal() {
    PyObject* m = PyModule_Create(&module);
    if (m && PyModule_AddStringConstant(m, "torch_version", PQ2_TORCH_VERSION) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
