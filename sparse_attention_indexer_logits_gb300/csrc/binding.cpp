// The serving operators' calls from Python (module _calls): the checks of the
// tensors and the calls of the C ABI, nothing else.  A decode step makes these
// calls every few microseconds of GPU time; through ctypes, with the checks in
// Python, a call took 7 to 25 us of host time, more than its kernels: the
// rotation of a step of 64 tokens into pages 13.3 us from Python, now 3.3, and
// 64 tokens over listed positions, waited for, 55 us, now 40.
//
// Every function takes the Python wrapper's arguments in order, positionally,
// raises ValueError for a tensor that does not fit, and returns the C call's
// code.
#include <Python.h>

#include <dlfcn.h>
#include <math.h>
#include <stdarg.h>

#include <exception>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "pml.h"

namespace {

// ------------------------------------------------------------------ the library

#define PML_CALLS(X) \
    X(pml_rope) X(pml_rope_append) X(pml_index_quant_append) X(pml_paged_attention) \
    X(pml_sparse_attention) X(pml_attention_workspace_bytes) X(pml_default_num_ctas) \
    X(pml_pages_fork) X(pml_pages_extend) X(pml_pages_free) X(pml_pages_compact) X(pml_pages_copy)

#define PML_MEMBER(name) decltype(&::name) name = nullptr;
struct Library {
    PML_CALLS(PML_MEMBER)
} pml;

// ------------------------------------------------------------------ arguments

struct Refused {};    // a Python error is set

[[noreturn]] void refuse(const char* format, ...)
{
    va_list args;
    va_start(args, format);
    PyErr_FormatV(PyExc_ValueError, format, args);
    va_end(args);
    throw Refused();
}

// The device of the call's tensors (-1: none seen yet).
thread_local int call_device = -1;

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
        throw Refused();
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.is_cuda()) {
        const int device = (int)t.get_device();
        if (call_device < 0) call_device = device;
        else if (device != call_device) refuse("%s must be on the device of the other tensors", name);
    }
    return t;
}

int narrow(int64_t v, const char* name)
{
    if (v != (int)v) refuse("%s is too large", name);
    return (int)v;
}

int integer(PyObject* o, const char* name)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Refused();
    return narrow(v, name);
}

float real(PyObject* o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Refused();
    return (float)v;
}

int truth(PyObject* o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Refused();
    return v;
}

// The call's stream, once its tensors have been seen: all of them, and the
// stream, belong to the current device (its properties, status word and
// workspace are what the library uses).
cudaStream_t stream_of(PyObject* o)
{
    const int current = c10::cuda::current_device();
    if (call_device >= 0 && call_device != current) refuse("the tensors must be on the current device");
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* index = PyObject_GetAttrString(o, "device_index");
    if (index) {
        const long long device = PyLong_AsLongLong(index);
        Py_DECREF(index);
        if (device == -1 && PyErr_Occurred()) throw Refused();
        if (device != current) refuse("stream must be of the current device");
    } else {
        PyErr_Clear();                            // a stand-in that has the handle alone
    }
    PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
    if (!raw) throw Refused();
    void* s = PyLong_AsVoidPtr(raw);
    Py_DECREF(raw);
    if (!s && PyErr_Occurred()) throw Refused();
    return static_cast<cudaStream_t>(s);
}

int dtype_code(at::ScalarType t)
{
    return t == at::kFloat ? PML_DTYPE_FLOAT32 : t == at::kBFloat16 ? PML_DTYPE_BFLOAT16
           : t == at::kHalf ? PML_DTYPE_FLOAT16 : -1;
}

// A [tokens, heads, dim] tensor with unit last stride.
struct Rows {
    void* data;
    int64_t token, head;
    int tokens, heads, dim;
    at::ScalarType type;

    bool same_shape(const Rows& o) const { return tokens == o.tokens && heads == o.heads && dim == o.dim; }
};

Rows rows_of(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (t.dim() != 3 || (t.stride(2) != 1 && t.size(2) > 1))
        refuse("%s must be [tokens, heads, dim] with unit last stride", name);
    return {t.data_ptr(), t.stride(0), t.stride(1), narrow(t.size(0), name), narrow(t.size(1), name),
            narrow(t.size(2), name), t.scalar_type()};
}

Rows rows_of(PyObject* o, const char* name, const Rows& like)
{
    const Rows r = rows_of(o, name);
    if (r.type != like.type) refuse("%s must have the type of the other rows", name);
    return r;
}

Rows output_of(PyObject* o, const char* name, const Rows& like, const char* like_name)
{
    const Rows r = rows_of(o, name, like);
    if (!r.same_shape(like)) refuse("%s must have %s's shape", name, like_name);
    return r;
}

void need_half(const Rows& q)
{
    if (q.type != at::kBFloat16 && q.type != at::kHalf) refuse("q must be bfloat16 or float16");
}

// A contiguous int32 tensor of `count` values (-1: any number).
int32_t* ints(PyObject* o, const char* name, int64_t count = -1)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || !t.is_cuda() || !t.is_contiguous())
        refuse("%s must be a contiguous CUDA int32 tensor", name);
    if (count >= 0 && t.numel() != count) refuse("%s must hold %lld values", name, (long long)count);
    return static_cast<int32_t*>(t.data_ptr());
}

int count_of(PyObject* o, const char* name) { return narrow(tensor(o, name).numel(), name); }

void* contiguous(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
    if (!t.is_contiguous()) refuse("%s must be contiguous", name);
    return t.data_ptr();
}

// An int32 [rows, width] tensor with unit last stride.
struct Table {
    int32_t* data;
    int64_t stride;
    int rows, width;
};

Table table_of(PyObject* o, const char* name)
{
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kInt || !t.is_cuda() || t.dim() != 2 || (t.stride(1) != 1 && t.size(1) > 1))
        refuse("%s must be a CUDA int32 [rows, width] tensor with unit last stride", name);
    return {static_cast<int32_t*>(t.data_ptr()), t.stride(0), narrow(t.size(0), name), narrow(t.size(1), name)};
}

// A [pages, 64, heads, dim] tensor with unit last stride.
struct Cache {
    void* data;
    int64_t page, slot, head, pages;
    int heads, dim;
};

Cache cache_of(PyObject* o, const char* name, const Rows& like)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda() || t.dim() != 4 || t.size(1) != 64 || (t.stride(3) != 1 && t.size(3) > 1))
        refuse("%s must be a CUDA [pages, 64, heads, dim] tensor with unit last stride", name);
    if (t.scalar_type() != like.type) refuse("%s must have the rows' type", name);
    return {t.data_ptr(), t.stride(0), t.stride(1), t.stride(2), t.size(0), narrow(t.size(2), name),
            narrow(t.size(3), name)};
}

// The two caches of a call on rows of `dim` elements.
struct Caches {
    Cache k, v;
};

Caches caches_of(PyObject* k_cache, PyObject* v_cache, const Rows& like)
{
    const Caches c = {cache_of(k_cache, "k_cache", like), cache_of(v_cache, "v_cache", like)};
    if (c.k.pages != c.v.pages || c.k.heads != c.v.heads || c.k.dim != c.v.dim || c.k.dim != like.dim)
        refuse("k_cache and v_cache must be [pages, 64, kv_heads, dim] with q's dim");
    return c;
}

struct Rotation {
    const void* positions;
    const void* freq;
    int positions_64, freq_64, dim;
};

Rotation rotation_of(PyObject* positions, PyObject* inv_freq, int64_t tokens)
{
    const at::Tensor& p = tensor(positions, "positions");
    const at::Tensor& f = tensor(inv_freq, "inv_freq");
    if ((p.scalar_type() != at::kInt && p.scalar_type() != at::kLong) || !p.is_cuda())
        refuse("positions must be a CUDA int32 or int64 tensor");
    if ((f.scalar_type() != at::kFloat && f.scalar_type() != at::kDouble) || !f.is_cuda())
        refuse("inv_freq must be a CUDA float32 or float64 tensor");
    if (!p.is_contiguous() || !f.is_contiguous()) refuse("positions and inv_freq must be contiguous");
    if (p.numel() != tokens) refuse("positions must hold one value per token");
    return {p.data_ptr(), f.data_ptr(), p.scalar_type() == at::kLong, f.scalar_type() == at::kDouble,
            narrow(2 * f.numel(), "inv_freq")};
}

// A call's own workspace: it may go back to its allocator when the call
// returns, since what takes its memory next on the stream runs after the kernels.
struct Workspace {
    void* data;
    int64_t bytes;
    bool own = false;

    Workspace(PyObject* o, int head_dim, cudaStream_t stream)
    {
        if (o != Py_None) {
            const at::Tensor& t = tensor(o, "workspace");
            if (!t.is_cuda() || !t.is_contiguous()) refuse("workspace must be a contiguous CUDA tensor");
            data = t.data_ptr();
            bytes = t.numel() * t.element_size();
            return;
        }
        static int ctas[64] = {};                 // by device
        const int device = c10::cuda::current_device();
        int n = device < 64 ? ctas[device] : 0;
        if (n == 0) {
            n = pml.pml_default_num_ctas(device);
            if (device < 64) ctas[device] = n;
        }
        bytes = pml.pml_attention_workspace_bytes(n, head_dim);
        if (bytes < 16) bytes = 16;               // the call refuses the head dimension
        data = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, stream);
        own = true;
    }
    Workspace(const Workspace&) = delete;
    ~Workspace()
    {
        if (own) c10::cuda::CUDACachingAllocator::raw_delete(data);
    }
};

// The call without the interpreter's lock; its code as a Python number.
template <class F>
PyObject* run(F call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// ------------------------------------------------------------------ the calls

PyObject* rope(PyObject* const* p)
{
    const Rows x = rows_of(p[0], "x");
    const int dtype = dtype_code(x.type);
    if (dtype < 0) refuse("x must be float32, bfloat16 or float16");
    const Rotation r = rotation_of(p[1], p[2], x.tokens);
    const Rows out = output_of(p[3], "out", x, "x");
    const int offset = integer(p[4], "rot_offset"), interleaved = truth(p[5]), gradient = truth(p[7]);
    const float mscale = real(p[6]);
    const cudaStream_t s = stream_of(p[8]);
    return run([&] {
        return pml.pml_rope(x.data, x.token, x.head, out.data, out.token, out.head, dtype, r.positions,
                            r.positions_64, r.freq, r.freq_64, r.dim, offset, interleaved, mscale, gradient,
                            x.tokens, x.heads, x.dim, s);
    });
}

PyObject* rope_append(PyObject* const* p)
{
    const Rows q = rows_of(p[0], "q");
    need_half(q);
    const Rows k = rows_of(p[1], "k", q), v = rows_of(p[2], "v", q);
    if (!v.same_shape(k) || k.tokens != q.tokens || k.dim != q.dim)
        refuse("k and v must be [tokens, kv_heads, dim] with q's tokens and dim");
    const Rotation r = rotation_of(p[3], p[5], q.tokens);
    const int32_t* requests = ints(p[4], "requests", q.tokens);
    const Table table = table_of(p[8], "block_table");
    const Caches c = caches_of(p[6], p[7], q);
    if (c.k.heads != k.heads) refuse("k_cache and v_cache must have k's heads");
    const Rows out = output_of(p[9], "q_out", q, "q");
    const int offset = integer(p[10], "rot_offset"), interleaved = truth(p[11]);
    const float mscale = real(p[12]);
    const cudaStream_t s = stream_of(p[13]);
    return run([&] {
        return pml.pml_rope_append(q.data, q.token, q.head, out.data, out.token, out.head, k.data, k.token,
                                   k.head, v.data, v.token, v.head, dtype_code(q.type), r.positions,
                                   r.positions_64, requests, table.rows, r.freq, r.freq_64, r.dim, offset,
                                   interleaved, mscale, c.k.data, c.k.page, c.k.slot, c.k.head, c.v.data,
                                   c.v.page, c.v.slot, c.v.head, c.k.pages, table.data, table.stride,
                                   table.width, q.tokens, q.heads, k.heads, q.dim, s);
    });
}

PyObject* index_quant_append(PyObject* const* p)
{
    const Rows q = rows_of(p[0], "q");
    if (q.type != at::kBFloat16 || q.dim != 128) refuse("q must be bfloat16 [tokens, heads, 128]");
    const Rotation r = rotation_of(p[3], p[5], q.tokens);
    auto per_head = [&](PyObject* o, const char* name) {
        const at::Tensor& t = tensor(o, name);
        if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != q.tokens || t.size(1) != q.heads)
            refuse("%s must be float32 [tokens, heads]", name);
        return static_cast<float*>(contiguous(o, name));
    };
    const float* weights = per_head(p[2], "weights");
    void* k = nullptr;
    int64_t k_stride = 0, blocks = 0;
    const int32_t* requests = nullptr;
    uint8_t* kv = nullptr;
    Table table = {nullptr, 0, 0, 0};
    if (p[1] != Py_None) {
        const at::Tensor& t = tensor(p[1], "k");
        if (!t.is_cuda() || t.scalar_type() != at::kBFloat16 || t.dim() != 2 || t.size(0) != q.tokens ||
            t.size(1) != 128 || t.stride(1) != 1)
            refuse("k must be a CUDA bfloat16 [tokens, 128] tensor with unit last stride");
        if (p[4] == Py_None || p[6] == Py_None || p[7] == Py_None)
            refuse("keys need requests, kv_fused and block_table");
        k = t.data_ptr();
        k_stride = t.stride(0);
        requests = ints(p[4], "requests", q.tokens);
        table = table_of(p[7], "block_table");
        const at::Tensor& f = tensor(p[6], "kv_fused");
        kv = static_cast<uint8_t*>(contiguous(p[6], "kv_fused"));
        if (f.scalar_type() != at::kByte || f.numel() % 8448)
            refuse("kv_fused must be uint8 and hold whole 8448-byte blocks");
        blocks = f.numel() / 8448;
    }
    const at::Tensor& out = tensor(p[8], "q_out");
    if (out.dim() != 3 || out.size(0) != q.tokens || out.size(1) != q.heads || out.size(2) != 128 ||
        out.element_size() != 1)
        refuse("q_out must be 1-byte [tokens, heads, 128]");
    uint8_t* q_out = static_cast<uint8_t*>(contiguous(p[8], "q_out"));
    float* w_out = per_head(p[9], "w_out");
    const float weight_scale = real(p[10]), mscale = real(p[13]);
    const int offset = integer(p[11], "rot_offset"), interleaved = truth(p[12]);
    const cudaStream_t s = stream_of(p[14]);
    return run([&] {
        return pml.pml_index_quant_append(q.data, q.token, q.head, k, k_stride, weights, weight_scale,
                                          r.positions, r.positions_64, requests, table.rows, r.freq,
                                          r.freq_64, r.dim, offset, interleaved, mscale, q_out, w_out, kv,
                                          blocks, table.data, table.stride, table.width, q.tokens, q.heads, s);
    });
}

// The checks that both attention calls share.
struct Attention {
    Rows q, out;
    Caches c;
    Table table;
    const int32_t* lens;
    float scale;
    float* lse = nullptr;

    Attention(PyObject* q_, PyObject* k_cache, PyObject* v_cache, PyObject* block_table, PyObject* kv_lens,
              PyObject* out_, PyObject* softmax_scale, PyObject* lse_)
        : q(rows_of(q_, "q"))
    {
        need_half(q);
        c = caches_of(k_cache, v_cache, q);
        table = table_of(block_table, "block_table");
        lens = ints(kv_lens, "kv_lens", table.rows);
        out = output_of(out_, "out", q, "q");
        scale = softmax_scale == Py_None ? (float)(1.0 / sqrt((double)(q.dim > 0 ? q.dim : 1)))
                                         : real(softmax_scale);
        if (lse_ != Py_None) {
            const at::Tensor& t = tensor(lse_, "lse");
            if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != q.tokens ||
                t.size(1) != q.heads || !t.is_contiguous() || !t.is_cuda())
                refuse("lse must be a contiguous CUDA float32 [tokens, heads] tensor");
            lse = static_cast<float*>(t.data_ptr());
        }
    }
};

PyObject* paged_attention(PyObject* const* p)
{
    const Attention a(p[0], p[1], p[2], p[3], p[4], p[6], p[7], p[10]);
    const int batch = a.table.rows;
    const int32_t* cu_q = nullptr;
    if (p[5] != Py_None) cu_q = ints(p[5], "cu_q", batch + 1LL);
    else if (batch == 0 ? a.q.tokens != 0 : a.q.tokens % batch != 0)
        refuse("without cu_q the tokens must divide equally over the requests");
    const int causal = truth(p[8]), window = integer(p[9], "window");
    const cudaStream_t s = stream_of(p[12]);
    const Workspace w(p[11], a.q.dim, s);
    return run([&] {
        return pml.pml_paged_attention(a.q.data, a.q.token, a.q.head, a.c.k.data, a.c.k.page, a.c.k.slot,
                                       a.c.k.head, a.c.v.data, a.c.v.page, a.c.v.slot, a.c.v.head,
                                       dtype_code(a.q.type), a.c.k.pages, a.table.data, a.table.stride,
                                       a.table.width, a.lens, cu_q, batch, a.q.tokens, a.q.heads,
                                       a.c.k.heads, a.q.dim, a.scale, causal, window, a.out.data,
                                       a.out.token, a.out.head, a.lse, w.data, w.bytes, s);
    });
}

PyObject* sparse_attention(PyObject* const* p)
{
    const Attention a(p[0], p[1], p[2], p[3], p[4], p[7], p[8], p[9]);
    const int32_t* requests = ints(p[5], "requests", a.q.tokens);
    const Table selected = table_of(p[6], "selected");
    if (selected.rows != a.q.tokens) refuse("selected must hold a row per token");
    const cudaStream_t s = stream_of(p[11]);
    const Workspace w(p[10], a.q.dim, s);
    return run([&] {
        return pml.pml_sparse_attention(a.q.data, a.q.token, a.q.head, a.c.k.data, a.c.k.page, a.c.k.slot,
                                        a.c.k.head, a.c.v.data, a.c.v.page, a.c.v.slot, a.c.v.head,
                                        dtype_code(a.q.type), a.c.k.pages, a.table.data, a.table.stride,
                                        a.table.width, a.lens, requests, a.table.rows, selected.data,
                                        selected.stride, selected.width, a.q.tokens, a.q.heads,
                                        a.c.k.heads, a.q.dim, a.scale, a.out.data, a.out.token,
                                        a.out.head, a.lse, w.data, w.bytes, s);
    });
}

struct Pool {
    int32_t* refs;
    int pages;
    Table table;
    int32_t* lens;

    Pool(PyObject* const* p)
        : refs(ints(p[0], "ref_counts")), pages(count_of(p[0], "ref_counts")), table(table_of(p[1], "block_table")),
          lens(ints(p[2], "seq_lens", table.rows))
    {
    }
};

PyObject* pages_fork(PyObject* const* p)
{
    const Pool o(p);
    const int32_t* parents = ints(p[3], "parents");
    const int n = count_of(p[3], "parents");
    const int32_t* children = ints(p[4], "children", n);
    int32_t *src = ints(p[5], "copy_src", n), *dst = ints(p[6], "copy_dst", n), *count = ints(p[7], "copy_count", 1);
    const cudaStream_t s = stream_of(p[8]);
    return run([&] {
        return pml.pml_pages_fork(o.refs, o.pages, o.table.data, o.table.stride, o.table.width, o.lens,
                                  o.table.rows, parents, children, n, src, dst, count, s);
    });
}

PyObject* pages_extend(PyObject* const* p)
{
    const Pool o(p);
    const int32_t* new_lens = ints(p[3], "new_lens", o.table.rows);
    int32_t* pages = ints(p[4], "new_pages");
    const int capacity = count_of(p[4], "new_pages");
    int32_t* count = ints(p[5], "new_count", 1);
    const cudaStream_t s = stream_of(p[6]);
    return run([&] {
        return pml.pml_pages_extend(o.refs, o.pages, o.table.data, o.table.stride, o.table.width, o.lens,
                                    o.table.rows, new_lens, pages, capacity, count, s);
    });
}

PyObject* pages_free(PyObject* const* p)
{
    const Pool o(p);
    const int32_t* list = ints(p[3], "rows");
    const int n = count_of(p[3], "rows");
    const cudaStream_t s = stream_of(p[4]);
    return run([&] {
        return pml.pml_pages_free(o.refs, o.pages, o.table.data, o.table.stride, o.table.width, o.lens,
                                  o.table.rows, list, n, s);
    });
}

PyObject* pages_compact(PyObject* const* p)
{
    const Pool o(p);
    int32_t* refs_out = ints(p[3], "ref_counts_out", o.pages);
    const Table out = table_of(p[4], "block_table_out");
    if (out.rows != o.table.rows || out.width != o.table.width)
        refuse("block_table_out must have block_table's shape");
    int32_t *remap = ints(p[5], "remap", o.pages), *src = ints(p[6], "copy_src");
    const int n = count_of(p[6], "copy_src");
    int32_t *dst = ints(p[7], "copy_dst", n), *count = ints(p[8], "copy_count", 1);
    const cudaStream_t s = stream_of(p[9]);
    return run([&] {
        return pml.pml_pages_compact(o.refs, o.pages, o.table.data, o.table.stride, o.table.width, o.lens,
                                     o.table.rows, refs_out, out.data, out.stride, remap, src, dst, n,
                                     count, s);
    });
}

PyObject* pages_copy(PyObject* const* p)
{
    const at::Tensor& t = tensor(p[0], "cache");
    const int at = truth(p[4]);                   // the dimension of the pages
    if (!t.is_cuda() || t.dim() <= at)
        refuse("cache must be a CUDA tensor [layers, pages, ...] or [pages, ...]");
    int64_t elems = 1;
    for (int64_t d = t.dim() - 1; d > at; --d) {
        if (t.size(d) > 1 && t.stride(d) != elems) refuse("each page of the cache must be contiguous");
        elems *= t.size(d);
    }
    const int64_t b = t.element_size();
    const int32_t* src = ints(p[1], "copy_src");
    const int n = count_of(p[1], "copy_src");
    const int32_t *dst = ints(p[2], "copy_dst", n), *count = ints(p[3], "copy_count", 1);
    const int layers = at ? narrow(t.size(0), "cache") : 1, pages = narrow(t.size(at), "cache");
    const cudaStream_t s = stream_of(p[5]);
    return run([&] {
        return pml.pml_pages_copy(t.data_ptr(), layers, at ? t.stride(0) * b : 0, pages, t.stride(at) * b,
                                  elems * b, src, dst, count, n, s);
    });
}

// ------------------------------------------------------------------ the module

// The entry points' addresses, from the loaded library's handle.
PyObject* bind(PyObject*, PyObject* handle)
{
    void* h = PyLong_AsVoidPtr(handle);
    if (!h && PyErr_Occurred()) return nullptr;
#define PML_BIND(name)                                                       \
    if (!(pml.name = reinterpret_cast<decltype(pml.name)>(dlsym(h, #name)))) \
        return PyErr_Format(PyExc_RuntimeError, "libpml.so lacks " #name);
    PML_CALLS(PML_BIND)
    Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n)
{
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments expected, not %zd", N, n);
    if (!pml.pml_rope) return PyErr_Format(PyExc_RuntimeError, "the library is not bound");
    call_device = -1;
    try {
        return F(args);
    } catch (const Refused&) {
        return nullptr;
    } catch (const std::exception&) {    // (the allocator's, with PyTorch's own types)
        torch::translate_exception_to_python(std::current_exception());
        return nullptr;
    }
}

#define PML_ENTRY(name, n) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<name, n>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {
    {"bind", bind, METH_O, nullptr},
    PML_ENTRY(rope, 9),
    PML_ENTRY(rope_append, 14),
    PML_ENTRY(index_quant_append, 15),
    PML_ENTRY(paged_attention, 13),
    PML_ENTRY(sparse_attention, 12),
    PML_ENTRY(pages_fork, 9),
    PML_ENTRY(pages_extend, 7),
    PML_ENTRY(pages_free, 5),
    PML_ENTRY(pages_compact, 10),
    PML_ENTRY(pages_copy, 6),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
