// serving_binding.cpp -- the Python side of the serving and norm calls: checks of
// tensors, allocation of outputs and workspaces, and the call into librope.
//
// A decode step makes these calls once or more per layer, each a few
// microseconds on the device.  Written in Python over ctypes, an attention call
// took 21 us of the host's time and cache_append 10, their launches included;
// here they take 8 to 10 and 2.6.  Like the Python binding it only marshals:
// every step runs in librope, whose entry points it is given by bind() (so that
// there is one library in the process, whichever file it came from).
#include <Python.h>

#include <algorithm>
#include <cstdint>
#include <initializer_list>
#include <memory>
#include <mutex>
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/function.h>
#include <torch/csrc/autograd/functions/basic_ops.h>
#include <torch/csrc/autograd/functions/utils.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/autograd/saved_variable.h>
#include <torch/csrc/autograd/variable.h>

#include "rope.h"

namespace {

decltype(&rope_cache_append) g_append = nullptr;
decltype(&rope_attention_packed_fwd) g_packed = nullptr;
decltype(&rope_attention_packed_workspace) g_packed_bytes = nullptr;
decltype(&rope_attention_decode_fwd) g_decode = nullptr;
decltype(&rope_attention_decode_workspace) g_decode_bytes = nullptr;
decltype(&rope_norm_qk_fwd) g_norm = nullptr;
decltype(&rope_norm_qk_bwd) g_norm_bwd = nullptr;
decltype(&rope_norm_qk_workspace) g_norm_bytes = nullptr;
decltype(&rope_norm_cache_append) g_norm_append = nullptr;
decltype(&rope_tables_build_scaled) g_tables_scaled = nullptr;
decltype(&rope_attention_paged_fwd) g_paged = nullptr;
decltype(&rope_attention_paged_workspace) g_paged_bytes = nullptr;

// A Python exception has been set.
struct PythonError {};

// Other Python threads run while the library launches: a launch waits when the
// stream's queue is full, and what it waits for may need the interpreter.
struct Unlocked {
    PyThreadState *s = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(s); }
};

[[noreturn]] void fail(PyObject *type, const std::string &what)
{
    PyErr_SetString(type, what.c_str());
    throw PythonError();
}

template <class F, class... A>
rope_status unlocked(F f, A... a)
{
    const Unlocked u;
    return f(a...);
}

std::string shape_of(const at::Tensor &t)
{
    std::string s = "[";
    for (int64_t i = 0; i < t.dim(); ++i)
        s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + "]";
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        fail(PyExc_TypeError, std::string(name) + ": expected a tensor, got " + Py_TYPE(o)->tp_name);
    return THPVariable_Unpack(o);
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PythonError();
    return v;
}

int32_t truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw PythonError();
    return v;
}

double number(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw PythonError();
    return v;
}

int32_t type16(const at::Tensor &t, const char *what)
{
    if (t.scalar_type() == at::kBFloat16)
        return ROPE_BF16;
    if (t.scalar_type() == at::kHalf)
        return ROPE_F16;
    fail(PyExc_TypeError, std::string(what) + " takes bf16 or fp16 tensors, got " + c10::toString(t.scalar_type()));
}

// One call: the device its tensors live on and the stream it runs on.
struct Call {
    c10::DeviceIndex device;
    cudaStream_t stream;
    bool own_stream;                           // not the current one

    Call(const at::Tensor &first, PyObject *s) : Call(cuda_index(first), s) {}

    static c10::DeviceIndex cuda_index(const at::Tensor &first)
    {
        if (!first.is_cuda())
            fail(PyExc_ValueError, "expected CUDA tensors, got one on " + first.device().str());
        return first.get_device();
    }

    Call(c10::DeviceIndex on, PyObject *s) : device(on)
    {
        const cudaStream_t current = c10::cuda::getCurrentCUDAStream(device).stream();
        stream = current;
        if (s != Py_None) {
            if (PyLong_Check(s)) {
                stream = reinterpret_cast<cudaStream_t>(integer(s));
            } else {
                PyObject *d = PyObject_GetAttrString(s, "device_index");
                if (d == nullptr)
                    throw PythonError();
                const long at = PyLong_AsLong(d);
                Py_DECREF(d);
                if (at == -1 && PyErr_Occurred())
                    throw PythonError();
                if (at != device)
                    fail(PyExc_ValueError, "the stream belongs to cuda:" + std::to_string(at) +
                                               ", the tensors to cuda:" + std::to_string((int)device));
                PyObject *h = PyObject_GetAttrString(s, "cuda_stream");
                if (h == nullptr)
                    throw PythonError();
                const long long v = PyLong_AsLongLong(h);
                Py_DECREF(h);
                if (v == -1 && PyErr_Occurred())
                    throw PythonError();
                stream = reinterpret_cast<cudaStream_t>(v);
            }
        }
        own_stream = stream != current;
    }

    void on_device(const at::Tensor &t, const char *name, at::ScalarType type) const
    {
        if (t.scalar_type() != type)
            fail(PyExc_ValueError, std::string(name) + " must be a " + c10::toString(type) + " tensor, got " +
                                       c10::toString(t.scalar_type()));
        if (!t.is_cuda() || t.get_device() != device)
            fail(PyExc_ValueError, std::string(name) + " must be on cuda:" + std::to_string((int)device) + ", got " +
                                       t.device().str());
    }

    // Address of a contiguous tensor of the type with n elements (-1: any), or
    // null for None where that is allowed.
    const void *dense(PyObject *o, const char *name, at::ScalarType type, int64_t n, bool optional = false) const
    {
        if (optional && o == Py_None)
            return nullptr;
        const at::Tensor &t = tensor(o, name);
        on_device(t, name, type);
        if (!t.is_contiguous())
            fail(PyExc_ValueError, std::string(name) + " must be contiguous");
        if (n >= 0 && (t.dim() != 1 || t.size(0) != n))
            fail(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(n) + "], got " + shape_of(t));
        return t.data_ptr();
    }

    const int32_t *ints(PyObject *o, const char *name, int64_t n, bool optional = false) const
    {
        return static_cast<const int32_t *>(dense(o, name, at::kInt, n, optional));
    }

    // A new tensor for the call, from the memory of the call's stream: the allocator
    // hands a block out as soon as the host has dropped it, to calls that run behind
    // its last use on the same stream.  A block of the current stream could still
    // be written by work queued there.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const
    {
        const at::TensorOptions options = at::TensorOptions().dtype(type).device(at::kCUDA, device);
        if (!own_stream)
            return at::empty(shape, options);
        const c10::cuda::CUDAStreamGuard guard(stream == nullptr
                                                   ? c10::cuda::getDefaultCUDAStream(device)
                                                   : c10::cuda::getStreamFromExternal(stream, device));
        return at::empty(shape, options);
    }

    // The same, for the caller, who uses it on the current stream next: once
    // dropped, it is handed out again when the work queued there is done.
    at::Tensor empty_returned(at::IntArrayRef shape, at::ScalarType type) const
    {
        at::Tensor t = empty(shape, type);
        if (own_stream)
            t.record_stream(c10::cuda::getCurrentCUDAStream(device).unwrap());
        return t;
    }

    // The workspace: the given tensor, or a new one (undefined: none needed).
    at::Tensor workspace(PyObject *given, int64_t need) const
    {
        if (given == Py_None)
            return need > 0 ? empty({need}, at::kByte) : at::Tensor();
        const at::Tensor &t = tensor(given, "workspace");
        if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
            fail(PyExc_ValueError, "workspace must be a contiguous tensor on cuda:" + std::to_string((int)device));
        return t;
    }
};

// A [tokens, heads, D] tensor, dense but for its tokens.
struct Rows {
    const void *p;
    int64_t n, stride;
    int32_t H, D;

    Rows(const Call &c, PyObject *o, const char *name, at::ScalarType type, int64_t heads = -1, int64_t d = -1)
    {
        const at::Tensor &t = tensor(o, name);
        c.on_device(t, name, type);
        if (t.dim() != 3 || (heads >= 0 && t.size(1) != heads) || (d >= 0 && t.size(2) != d))
            fail(PyExc_ValueError, std::string(name) + " must be [tokens, " +
                                       (heads >= 0 ? std::to_string(heads) : std::string("heads")) + ", " +
                                       (d >= 0 ? std::to_string(d) : std::string("D")) + "], got " + shape_of(t));
        n = t.size(0);
        if (t.size(1) > INT32_MAX || t.size(2) > INT32_MAX)
            fail(PyExc_ValueError, std::string(name) + " is too large: " + shape_of(t));
        H = (int32_t)t.size(1);
        D = (int32_t)t.size(2);
        if (t.numel() > 0 && ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D)))
            fail(PyExc_ValueError, std::string(name) + ": heads and features must be dense");
        stride = n > 1 ? t.stride(0) : (int64_t)H * D;
        p = t.data_ptr();
    }
};

struct Tables {
    const float *cos, *sin;
    int64_t rows;
    int32_t rotary_dim;

    Tables(const Call &c, PyObject *cs, PyObject *sn, PyObject *rd)
    {
        const at::Tensor &a = tensor(cs, "cos"), &b = tensor(sn, "sin");
        if (a.dim() != 2 || a.sizes() != b.sizes())
            fail(PyExc_ValueError, "cos and sin must be [rows, rotary_dim / 2] tables of the same shape");
        rows = a.size(0);
        if (a.size(1) > INT32_MAX / 2 || (rd != Py_None && integer(rd) != 2 * a.size(1)))
            fail(PyExc_ValueError, "table width " + std::to_string(a.size(1)) + " does not match rotary_dim");
        rotary_dim = (int32_t)(2 * a.size(1));
        cos = static_cast<const float *>(c.dense(cs, "cos", at::kFloat, -1));
        sin = static_cast<const float *>(c.dense(sn, "sin", at::kFloat, -1));
    }
};

struct Cache {
    void *k, *v;
    int64_t n_pages;
    int32_t Hk, page, D;

    Cache(const Call &c, PyObject *ko, PyObject *vo, at::ScalarType type)
    {
        const at::Tensor &a = tensor(ko, "k_pages"), &b = tensor(vo, "v_pages");
        if (a.dim() != 4 || a.sizes() != b.sizes() || a.size(1) > INT32_MAX || a.size(2) > INT32_MAX ||
            a.size(3) > INT32_MAX)
            fail(PyExc_ValueError, "k_pages and v_pages must be [pages, Hk, page_size, D] of one shape");
        k = const_cast<void *>(c.dense(ko, "k_pages", type, -1));
        v = const_cast<void *>(c.dense(vo, "v_pages", type, -1));
        n_pages = a.size(0);
        Hk = (int32_t)a.size(1);
        page = (int32_t)a.size(2);
        D = (int32_t)a.size(3);
    }
};

// The output: the given tensor of that shape, or a new one.
at::Tensor output(const Call &c, PyObject *given, const Rows &like, at::ScalarType type, const char *name = "out")
{
    if (given == Py_None)
        return c.empty_returned({like.n, like.H, like.D}, type);
    const at::Tensor &t = tensor(given, name);
    c.dense(given, name, type, -1);
    if (t.dim() != 3 || t.size(0) != like.n || t.size(1) != like.H || t.size(2) != like.D)
        fail(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(like.n) + ", " + std::to_string(like.H) + ", " +
                                   std::to_string(like.D) + "], got " + shape_of(t));
    return t;
}

// Tells autograd that a tensor the caller holds has been written, as torch's own
// in-place operations do: a graph that saved it then refuses to run backward.
void written(const at::Tensor &t)
{
    if (!t.is_inference())                     // (these have no version)
        t.unsafeGetTensorImpl()->bump_version();
}

void expect(Py_ssize_t got, Py_ssize_t want)
{
    if (got != want)
        fail(PyExc_TypeError, "expected " + std::to_string(want) + " arguments");
    if (g_append == nullptr)
        fail(PyExc_RuntimeError, "bind() comes first");
}

PyObject *status(rope_status st) { return PyLong_FromLong(st); }

// bind(addresses of the entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    constexpr int kEntries = 12;
    if (n != kEntries) {
        PyErr_Format(PyExc_TypeError, "expected %d addresses", kEntries);
        return nullptr;
    }
    void *p[kEntries];
    for (int i = 0; i < kEntries; ++i) {
        p[i] = PyLong_AsVoidPtr(a[i]);
        if (p[i] == nullptr) {
            if (!PyErr_Occurred())
                PyErr_SetString(PyExc_ValueError, "a null address");
            return nullptr;
        }
    }
    g_append = reinterpret_cast<decltype(g_append)>(p[0]);
    g_packed = reinterpret_cast<decltype(g_packed)>(p[1]);
    g_packed_bytes = reinterpret_cast<decltype(g_packed_bytes)>(p[2]);
    g_decode = reinterpret_cast<decltype(g_decode)>(p[3]);
    g_decode_bytes = reinterpret_cast<decltype(g_decode_bytes)>(p[4]);
    g_norm = reinterpret_cast<decltype(g_norm)>(p[5]);
    g_norm_bwd = reinterpret_cast<decltype(g_norm_bwd)>(p[6]);
    g_norm_bytes = reinterpret_cast<decltype(g_norm_bytes)>(p[7]);
    g_norm_append = reinterpret_cast<decltype(g_norm_append)>(p[8]);
    g_tables_scaled = reinterpret_cast<decltype(g_tables_scaled)>(p[9]);
    g_paged = reinterpret_cast<decltype(g_paged)>(p[10]);
    g_paged_bytes = reinterpret_cast<decltype(g_paged_bytes)>(p[11]);
    Py_RETURN_NONE;
}

// cache_append(k, v, k_pages, v_pages, block_table, cu_seqlens, cache_lens, cos,
//              sin, pos, pos_offset, rotary_dim, layout, stream) -> status
PyObject *cache_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 14);
        const at::Tensor &k = tensor(a[0], "k");
        const Call c(k, a[13]);
        const int32_t code = type16(k, "cache_append");
        const at::ScalarType type = k.scalar_type();
        const Cache pool(c, a[2], a[3], type);
        const Rows kr(c, a[0], "k", type, pool.Hk, pool.D), vr(c, a[1], "v", type, pool.Hk, pool.D);
        if (kr.n != vr.n)
            fail(PyExc_ValueError, "k and v must have the same tokens");
        const at::Tensor &table = tensor(a[4], "block_table");
        if (table.dim() != 2)
            fail(PyExc_ValueError, "block_table must be [n_seqs, max_blocks], got " + shape_of(table));
        const int64_t seqs = table.size(0), blocks = table.size(1);
        const Tables t(c, a[7], a[8], a[11]);
        const int32_t *list = c.ints(a[4], "block_table", -1);
        const c10::cuda::CUDAGuard guard(c.device);
        const rope_status st =
            unlocked(g_append, kr.p, vr.p, pool.k, pool.v, list, c.ints(a[5], "cu_seqlens", seqs + 1),
                     c.ints(a[6], "cache_lens", seqs), t.cos, t.sin, c.ints(a[9], "pos", kr.n, true), integer(a[10]),
                     seqs, kr.n, kr.stride, vr.stride, pool.Hk, pool.D, t.rotary_dim, (int32_t)integer(a[12]),
                     pool.page, pool.n_pages, blocks, code, t.rows, c.stream);
        if (st == ROPE_OK) {
            written(tensor(a[2], "k_pages"));
            written(tensor(a[3], "v_pages"));
        }
        return status(st);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// attention_packed(q, k, v, cu_seqlens_q, cos, sin, cu_seqlens_k, pos_q, pos_k,
//                  rotary_dim, layout, causal, scale, out, workspace, stream)
// -> the output, or a status
PyObject *attention_packed(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 16);
        const at::Tensor &q = tensor(a[0], "q");
        const Call c(q, a[15]);
        const int32_t code = type16(q, "attention_packed");
        const at::ScalarType type = q.scalar_type();
        const Rows qr(c, a[0], "q", type), kr(c, a[1], "k", type, -1, qr.D), vr(c, a[2], "v", type, kr.H, qr.D);
        if (kr.n != vr.n)
            fail(PyExc_ValueError, "k and v must have the same tokens");
        const at::Tensor &cu = tensor(a[3], "cu_seqlens_q");
        if (cu.dim() != 1 || cu.size(0) < 1)
            fail(PyExc_ValueError, "cu_seqlens_q must be [n_seqs + 1], got " + shape_of(cu));
        const int64_t seqs = cu.size(0) - 1;
        const int32_t *cuq = c.ints(a[3], "cu_seqlens_q", seqs + 1);
        const int32_t *cuk = a[6] == Py_None ? cuq : c.ints(a[6], "cu_seqlens_k", seqs + 1);
        const Tables t(c, a[4], a[5], a[9]);
        const int32_t *pq = c.ints(a[7], "pos_q", qr.n, true), *pk = c.ints(a[8], "pos_k", kr.n, true);
        const int32_t layout = (int32_t)integer(a[10]), causal = truth(a[11]);
        const float scale = a[12] == Py_None ? -1.0f : (float)number(a[12]);
        const int64_t need = g_packed_bytes(seqs, qr.n, kr.n, qr.H, kr.H, qr.D);
        // (sizes without a workspace are refused by the call, which says why)
        const c10::cuda::CUDAGuard guard(c.device);
        const at::Tensor out = output(c, a[13], qr, type), ws = c.workspace(a[14], need);
        const rope_status st =
            unlocked(g_packed, qr.p, kr.p, vr.p, out.data_ptr(), t.cos, t.sin, pq, pk, cuq, cuk, seqs, qr.n, kr.n, qr.stride,
                     kr.stride, vr.stride, qr.H, kr.H, qr.D, t.rotary_dim, layout, causal, scale, code, t.rows,
                     ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (int64_t)ws.nbytes() : 0, c.stream);
        if (st != ROPE_OK)
            return status(st);
        if (a[13] != Py_None)
            written(out);
        return THPVariable_Wrap(out);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// attention_shared_prefix(q, k_pages, v_pages, block_table, seq_lens,
//     prefix_table, prefix_len, cos, sin, pos_q, rotary_dim, layout, scale, out,
//     workspace, stream) -> the output, or a status
PyObject *attention_shared_prefix(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 16);
        const at::Tensor &q = tensor(a[0], "q");
        const Call c(q, a[15]);
        const int32_t code = type16(q, "attention_shared_prefix");
        const at::ScalarType type = q.scalar_type();
        const Rows qr(c, a[0], "q", type);
        const Cache pool(c, a[1], a[2], type);
        if (pool.D != qr.D)
            fail(PyExc_ValueError, "the cache holds heads of " + std::to_string(pool.D) + " features, q of " +
                                       std::to_string(qr.D));
        const at::Tensor &table = tensor(a[3], "block_table");
        if (table.dim() != 2 || table.size(0) != qr.n)
            fail(PyExc_ValueError, "block_table must be [" + std::to_string(qr.n) + ", max_blocks], got " +
                                       shape_of(table));
        const int64_t blocks = table.size(1), prefix = integer(a[6]);
        const int32_t *list = c.ints(a[3], "block_table", -1), *lens = c.ints(a[4], "seq_lens", qr.n);
        const int32_t *pages = c.ints(a[5], "prefix_table", -1, true);
        if (prefix > 0 && (a[5] == Py_None || THPVariable_Unpack(a[5]).numel() < (prefix - 1) / std::max(pool.page, 1) + 1))
            fail(PyExc_ValueError, "prefix_table must name the pages of " + std::to_string(prefix) + " keys");
        const Tables t(c, a[7], a[8], a[10]);
        const int32_t *pq = c.ints(a[9], "pos_q", qr.n, true);
        const int32_t layout = (int32_t)integer(a[11]);
        const float scale = a[12] == Py_None ? -1.0f : (float)number(a[12]);
        const int64_t need = g_decode_bytes(qr.n, qr.H, pool.Hk, qr.D, pool.page, blocks, prefix);
        // (sizes without a workspace are refused by the call, which says why)
        const c10::cuda::CUDAGuard guard(c.device);
        const at::Tensor out = output(c, a[13], qr, type);
        const at::Tensor ws = c.workspace(a[14], need);
        const rope_status st =
            unlocked(g_decode, qr.p, pool.k, pool.v, out.data_ptr(), list, lens, pages, prefix, t.cos, t.sin, pq, qr.n,
                     qr.stride, qr.H, pool.Hk, qr.D, t.rotary_dim, layout, scale, pool.page, pool.n_pages, blocks,
                     code, t.rows, ws.defined() ? ws.data_ptr() : nullptr,
                     ws.defined() ? (int64_t)ws.nbytes() : 0, c.stream);
        if (st != ROPE_OK)
            return status(st);
        if (a[13] != Py_None)
            written(out);
        return THPVariable_Wrap(out);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// attention_paged(q, k_pages, v_pages, block_table, cu_seqlens_q, seq_lens, cos, sin,
//     pos_q, rotary_dim, layout, causal, scale, out, workspace, stream)
// -> the output, or a status
PyObject *attention_paged(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 16);
        const at::Tensor &q = tensor(a[0], "q");
        const Call c(q, a[15]);
        const int32_t code = type16(q, "attention_paged");
        const at::ScalarType type = q.scalar_type();
        const Rows qr(c, a[0], "q", type);
        const Cache pool(c, a[1], a[2], type);
        if (pool.D != qr.D)
            fail(PyExc_ValueError, "the cache holds heads of " + std::to_string(pool.D) + " features, q of " +
                                       std::to_string(qr.D));
        const at::Tensor &table = tensor(a[3], "block_table");
        if (table.dim() != 2)
            fail(PyExc_ValueError, "block_table must be [n_seqs, max_blocks], got " + shape_of(table));
        const int64_t seqs = table.size(0), blocks = table.size(1);
        const int32_t *list = c.ints(a[3], "block_table", -1), *cu = c.ints(a[4], "cu_seqlens_q", seqs + 1),
                      *lens = c.ints(a[5], "seq_lens", seqs), *pq = c.ints(a[8], "pos_q", qr.n, true);
        if ((a[6] == Py_None) != (a[7] == Py_None))
            fail(PyExc_ValueError, "cos and sin are given together, or neither");
        const float *cos = nullptr, *sin = nullptr;
        int64_t rows = 0;
        int32_t rotary_dim = 0;
        if (a[6] != Py_None) {
            const Tables t(c, a[6], a[7], a[9]);
            cos = t.cos;
            sin = t.sin;
            rows = t.rows;
            rotary_dim = t.rotary_dim;
            if (cos == nullptr || sin == nullptr)          // (an empty table is not a missing one)
                fail(PyExc_ValueError, "cos and sin must have rows");
        }
        const int32_t layout = (int32_t)integer(a[10]), causal = truth(a[11]);
        const float scale = a[12] == Py_None ? -1.0f : (float)number(a[12]);
        const int64_t need = g_paged_bytes(seqs, qr.n, qr.H, pool.Hk, qr.D, pool.page, blocks);
        // (sizes without a workspace are refused by the call, which says why)
        const c10::cuda::CUDAGuard guard(c.device);
        const at::Tensor out = output(c, a[13], qr, type), ws = c.workspace(a[14], need);
        const rope_status st =
            unlocked(g_paged, qr.p, pool.k, pool.v, out.data_ptr(), list, cu, lens, cos, sin, pq, seqs, qr.n, qr.stride, qr.H,
                     pool.Hk, qr.D, rotary_dim, layout, causal, scale, pool.page, pool.n_pages, blocks, code, rows,
                     ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (int64_t)ws.nbytes() : 0, c.stream);
        if (st != ROPE_OK)
            return status(st);
        if (a[13] != Py_None)
            written(out);
        return THPVariable_Wrap(out);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// A weight of the norm: a [D] tensor, in fp32 or the rows' type, or None.
struct Weight {
    const void *p = nullptr;
    at::ScalarType type = at::kFloat;
    bool given = false;

    Weight(const Call &c, PyObject *o, const char *name, at::ScalarType rows, int64_t D)
    {
        if (o == Py_None)
            return;
        const at::Tensor &t = tensor(o, name);
        given = true;
        type = t.scalar_type();
        if (type != at::kFloat && type != rows)
            fail(PyExc_ValueError, std::string(name) + " must be fp32 or of the rows' type, got " + c10::toString(type));
        p = c.dense(o, name, type, D);
    }
};

int32_t weight_code(const Weight &q, const Weight &k, int32_t rows)
{
    if (q.given && k.given && q.type != k.type)
        fail(PyExc_ValueError, "wq and wk must be of one type");
    return (q.given ? q.type : k.type) == at::kFloat ? ROPE_F32 : rows;
}

int32_t type_code(const at::Tensor &t, const char *what)
{
    return t.scalar_type() == at::kFloat ? ROPE_F32 : type16(t, what);
}

// A [B, H, S, D] or [B, S, H, D] tensor with dense features, or None.
struct Heads {
    const void *p = nullptr;
    int64_t B = 0, S = 0, strides[3] = {0, 0, 0};
    int32_t H = 0, D = 0;

    Heads(const Call &c, PyObject *o, const char *name, at::ScalarType type, bool seq_first)
    {
        if (o == Py_None)
            return;
        const at::Tensor &t = tensor(o, name);
        c.on_device(t, name, type);
        if (t.dim() != 4)
            fail(PyExc_ValueError, std::string(name) + " must be 4-dimensional, got " + shape_of(t));
        const int s = seq_first ? 1 : 2, h = seq_first ? 2 : 1;
        if (t.size(h) > INT32_MAX || t.size(3) > INT32_MAX)
            fail(PyExc_ValueError, std::string(name) + " is too large: " + shape_of(t));
        if (t.numel() > 0 && t.size(3) > 1 && t.stride(3) != 1)
            fail(PyExc_ValueError, std::string(name) + ": features must be dense");
        B = t.size(0);
        S = t.size(s);
        H = (int32_t)t.size(h);
        D = (int32_t)t.size(3);
        strides[0] = t.stride(0);
        strides[1] = t.stride(s);
        strides[2] = t.stride(h);
        p = t.data_ptr();
    }
};

// The sizes that queries and keys share, and their positions.
struct NormShape {
    int64_t B, S, pos_stride = 0;
    int32_t D;
    const int32_t *pos = nullptr;

    NormShape(const Call &c, const Heads &q, const Heads &k, bool has_q, bool has_k, PyObject *positions)
    {
        const Heads &x = has_q ? q : k;
        B = x.B;
        S = x.S;
        D = x.D;
        if (has_q && has_k && (q.B != k.B || q.S != k.S || q.D != k.D))
            fail(PyExc_ValueError, "q and k must agree in batch, sequence and head_dim");
        if (positions == Py_None)
            return;
        const at::Tensor &t = tensor(positions, "pos_idx");
        pos = c.ints(positions, "pos_idx", -1);
        if (t.dim() == 2 && t.size(0) == B && t.size(1) >= S)
            pos_stride = t.size(1);
        else if (t.dim() != 1 || t.size(0) != S)
            fail(PyExc_ValueError, "pos_idx must be [S] or [B, >=S], got " + shape_of(t));
        if (S == 0)
            pos_stride = 0;
    }
};

// The given tensor, dense and of the shape of `like`, or a new one.
at::Tensor like_or_new(const Call &c, PyObject *given, const char *name, const at::Tensor &like)
{
    if (given == Py_None)
        return c.empty_returned(like.sizes(), like.scalar_type());
    const at::Tensor &t = tensor(given, name);
    c.dense(given, name, like.scalar_type(), -1);
    if (t.sizes() != like.sizes())
        fail(PyExc_ValueError, std::string(name) + " must be " + shape_of(like) + ", got " + shape_of(t));
    return t;
}

PyObject *wrapped(const at::Tensor &t)
{
    if (!t.defined())
        Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *tuple_of(std::initializer_list<at::Tensor> ts)
{
    PyObject *r = PyTuple_New((Py_ssize_t)ts.size());
    if (r == nullptr)
        throw PythonError();
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts) {
        PyObject *o = wrapped(t);
        if (o == nullptr) {
            Py_DECREF(r);
            throw PythonError();
        }
        PyTuple_SET_ITEM(r, i++, o);
    }
    return r;
}

// norm_rotate_qk(q, k, wq, wk, cos, sin, eps, pos_idx, rotary_dim, layout,
//                seq_before_head, q_out, k_out, stream) -> (q_out, k_out), or a status
PyObject *norm_rotate_qk(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 14);
        const bool has_q = a[0] != Py_None, has_k = a[1] != Py_None;
        const at::Tensor &x = has_q ? tensor(a[0], "q") : tensor(a[1], "q or k");
        const Call c(x, a[13]);
        const int32_t code = type_code(x, "norm_rotate_qk"), seq_first = truth(a[10]);
        const at::ScalarType type = x.scalar_type();
        const Heads q(c, a[0], "q", type, seq_first), k(c, a[1], "k", type, seq_first);
        const NormShape z(c, q, k, has_q, has_k, a[7]);
        const Weight wq(c, a[2], "wq", type, z.D), wk(c, a[3], "wk", type, z.D);
        const Tables t(c, a[4], a[5], a[8]);
        const c10::cuda::CUDAGuard guard(c.device);
        const at::Tensor qo = has_q ? like_or_new(c, a[11], "q_out", tensor(a[0], "q")) : at::Tensor();
        const at::Tensor ko = has_k ? like_or_new(c, a[12], "k_out", tensor(a[1], "k")) : at::Tensor();
        const rope_status st =
            unlocked(g_norm, q.p, k.p, has_q ? qo.data_ptr() : nullptr, has_k ? ko.data_ptr() : nullptr, wq.p, wk.p, t.cos,
                     t.sin, z.pos, z.pos_stride, z.B, q.H, k.H, z.S, z.D, q.strides, k.strides, t.rotary_dim,
                     (int32_t)integer(a[9]), seq_first, (float)number(a[6]), code, weight_code(wq, wk, code), t.rows, c.stream);
        if (st != ROPE_OK)
            return status(st);
        if (has_q && a[11] != Py_None)
            written(qo);
        if (has_k && a[12] != Py_None)
            written(ko);
        return tuple_of({qo, ko});
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// norm_rotate_qk_backward(gq, gk, q, k, wq, wk, cos, sin, eps, pos_idx, rotary_dim,
//     layout, seq_before_head, want_wq, want_wk, stream) -> (dq, dk, dwq, dwk), or a status
PyObject *norm_rotate_qk_backward(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 16);
        const bool has_q = a[2] != Py_None, has_k = a[3] != Py_None;
        const at::Tensor &x = has_q ? tensor(a[2], "q") : tensor(a[3], "q or k");
        const Call c(x, a[15]);
        const int32_t code = type_code(x, "norm_rotate_qk_backward"), seq_first = truth(a[12]);
        const at::ScalarType type = x.scalar_type();
        const Heads q(c, a[2], "q", type, seq_first), k(c, a[3], "k", type, seq_first);
        const NormShape z(c, q, k, has_q, has_k, a[9]);
        const Weight wq(c, a[4], "wq", type, z.D), wk(c, a[5], "wk", type, z.D);
        const Tables t(c, a[6], a[7], a[10]);
        const void *gp[2] = {nullptr, nullptr};
        for (int i = 0; i < 2; ++i) {
            if (i == 0 ? !has_q : !has_k)
                continue;
            gp[i] = c.dense(a[i], i ? "gk" : "gq", type, -1);
            if (tensor(a[i], "gq").sizes() != tensor(a[2 + i], "q").sizes())
                fail(PyExc_ValueError, std::string(i ? "gk" : "gq") + " must be " + shape_of(tensor(a[2 + i], "q")) + ", got " +
                                           shape_of(tensor(a[i], "gq")));
        }
        const c10::cuda::CUDAGuard guard(c.device);
        at::Tensor d[4];
        for (int i = 0; i < 2; ++i) {
            if (i == 0 ? !has_q : !has_k)
                continue;
            d[i] = c.empty_returned(tensor(a[2 + i], "q").sizes(), type);
            const Weight &w = i ? wk : wq;
            if (truth(a[13 + i]) && w.given)
                d[2 + i] = c.empty_returned({z.D}, w.type);
        }
        auto at_of = [&](int i) { return d[i].defined() ? d[i].data_ptr() : nullptr; };
        const at::Tensor ws = c.workspace(Py_None, d[2].defined() || d[3].defined() ? g_norm_bytes(z.D) : 0);
        const rope_status st =
            unlocked(g_norm_bwd, q.p, k.p, gp[0], gp[1], at_of(0), at_of(1), wq.p, wk.p, at_of(2), at_of(3), t.cos, t.sin,
                     z.pos, z.pos_stride, z.B, q.H, k.H, z.S, z.D, q.strides, k.strides, t.rotary_dim, (int32_t)integer(a[11]),
                     seq_first, (float)number(a[8]), code, weight_code(wq, wk, code), t.rows,
                     ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? (int64_t)ws.nbytes() : 0, c.stream);
        if (st != ROPE_OK)
            return status(st);
        return tuple_of({d[0], d[1], d[2], d[3]});
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// norm_rotary_qk: the same calls as a node of torch's autograd.  In C++, because a
// training step makes them once a layer: with a Python node, forward and backward of
// a small layer took 200 us of the host's time.

int32_t dtype_code(at::ScalarType t)
{
    return t == at::kFloat ? ROPE_F32 : t == at::kBFloat16 ? ROPE_BF16 : ROPE_F16;
}

void *address(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// What both directions need of queries and keys that the forward call has checked.
struct NormSizes {
    int64_t B = 0, S = 0, strides[2][3] = {}, pos_stride = 0, rows = 0;
    int32_t H[2] = {0, 0}, D = 0, code = 0, w_code = ROPE_F32, rotary_dim = 0;

    NormSizes(const at::Tensor (&x)[2], const at::Tensor (&w)[2], const at::Tensor &cos, const at::Tensor &pos, bool seq_first)
    {
        const int s = seq_first ? 1 : 2, h = seq_first ? 2 : 1;
        for (int i = 0; i < 2; ++i) {
            if (w[i].defined())
                w_code = dtype_code(w[i].scalar_type());
            const at::Tensor &t = x[i];
            if (!t.defined())
                continue;
            B = t.size(0);
            S = t.size(s);
            H[i] = (int32_t)t.size(h);
            D = (int32_t)t.size(3);
            code = dtype_code(t.scalar_type());
            strides[i][0] = t.stride(0);
            strides[i][1] = t.stride(s);
            strides[i][2] = t.stride(h);
        }
        if (pos.defined() && pos.dim() == 2 && S > 0)
            pos_stride = pos.size(1);
        rows = cos.size(0);
        rotary_dim = (int32_t)(2 * cos.size(1));
    }
};

// Whether the library takes a tensor's strides: dense features, whole 16-byte vectors.
bool whole_vectors(const at::Tensor &t)
{
    const int64_t v = 16 / t.element_size();
    if (reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0 || (t.size(3) > 1 && t.stride(3) != 1))
        return false;
    for (int i = 0; i < 3; ++i)
        if (t.size(i) > 1 && (t.stride(i) <= 0 || t.stride(i) % v != 0))
            return false;
    return true;
}

// t, dense and 16-byte aligned.
at::Tensor dense_vectors(const at::Tensor &t)
{
    const at::Tensor d = t.contiguous();
    return reinterpret_cast<uintptr_t>(d.data_ptr()) % 16 == 0 ? d : d.clone();
}

// The backward node: queries, keys and weights (undefined: None), the tables and positions.
struct NormRotaryBackward : torch::autograd::Node {
    torch::autograd::SavedVariable saved[7];   // q, k, wq, wk, cos, sin, pos_idx
    bool given[7] = {};
    double eps = 0.0;
    int32_t layout = 0;
    bool seq_first = false;

    std::string name() const override { return "NormRotaryBackward"; }

    void release_variables() override
    {
        const std::lock_guard<std::mutex> lock(mutex_);
        for (auto &v : saved)
            v.reset_data();
    }

    torch::autograd::variable_list apply(torch::autograd::variable_list &&grads) override
    {
        const std::lock_guard<std::mutex> lock(mutex_);
        const auto self = shared_from_this();
        auto unpacked = [&](int i) { return given[i] ? saved[i].unpack(self) : at::Tensor(); };
        const at::Tensor cos = unpacked(4), sin = unpacked(5), pos = unpacked(6);
        at::Tensor x[2], w[2], g[2], dx[2], dw[2];
        // an output that took no part in the loss has no gradient, and an input (and weight)
        // that needs none is left out
        int next = 0;
        for (int i = 0; i < 2; ++i) {
            if (!given[i])
                continue;
            const at::Tensor &up = grads[next++];
            if (!up.defined() || !(task_should_compute_output(i) || task_should_compute_output(2 + i)))
                continue;
            x[i] = unpacked(i);
            w[i] = unpacked(2 + i);
            g[i] = dense_vectors(up);
            dx[i] = at::empty(x[i].sizes(), x[i].options().memory_format(at::MemoryFormat::Contiguous));
            if (w[i].defined() && task_should_compute_output(2 + i))
                dw[i] = at::empty({x[i].size(3)}, w[i].options());
        }
        torch::autograd::variable_list out(4);
        if (x[0].defined() || x[1].defined()) {
            const NormSizes z(x, w, cos, pos, seq_first);
            const c10::cuda::CUDAGuard guard(cos.get_device());
            at::Tensor ws;
            if (dw[0].defined() || dw[1].defined())
                ws = at::empty({g_norm_bytes(z.D)}, cos.options().dtype(at::kByte));
            const rope_status st =
                g_norm_bwd(address(x[0]), address(x[1]), address(g[0]), address(g[1]), address(dx[0]), address(dx[1]),
                           address(w[0]), address(w[1]), address(dw[0]), address(dw[1]), cos.const_data_ptr<float>(),
                           sin.const_data_ptr<float>(), static_cast<const int32_t *>(address(pos)), z.pos_stride, z.B, z.H[0],
                           z.H[1], z.S, z.D, z.strides[0], z.strides[1], z.rotary_dim, layout, seq_first, (float)eps, z.code,
                           z.w_code, z.rows, address(ws), ws.defined() ? (int64_t)ws.nbytes() : 0,
                           c10::cuda::getCurrentCUDAStream(cos.get_device()).stream());
            TORCH_CHECK(st == ROPE_OK, "rope_norm_qk_bwd: status ", (int)st);
        }
        for (int i = 0; i < 2; ++i) {
            if (task_should_compute_output(i))
                out[i] = dx[i];
            out[2 + i] = dw[i];
        }
        if (at::GradMode::is_enabled()) {
            // differentiable once: a second derivative through these is an error, not a zero
            for (at::Tensor &t : out)
                if (t.defined())
                    t = (*std::make_shared<torch::autograd::DelayedError>(
                        "norm_rotary_qk: its gradients cannot be differentiated", 1))({t.detach().set_requires_grad(true)})[0];
        }
        return out;
    }
};

// The forward call on checked arguments, and its node where a gradient is wanted.
rope_status norm_rotary_forward(const at::Tensor (&in)[7], double eps, int32_t layout, bool seq_first, at::Tensor (&y)[2])
{
    at::Tensor x[2] = {in[0], in[1]}, w[2] = {in[2], in[3]};
    const at::Tensor &cos = in[4], &sin = in[5], &pos = in[6];
    bool graph = false;
    for (int i = 0; i < 4 && at::GradMode::is_enabled(); ++i)
        graph = graph || (in[i].defined() && in[i].requires_grad());
    {
        const at::AutoGradMode off(false);
        for (int i = 0; i < 2; ++i)
            if (x[i].defined()) {
                if (!whole_vectors(x[i]))
                    x[i] = x[i].clone(at::MemoryFormat::Contiguous);
                y[i] = at::empty(x[i].sizes(), x[i].options().memory_format(at::MemoryFormat::Contiguous));
            }
        for (at::Tensor &t : w)                // (a weight may lie anywhere in a buffer of parameters)
            if (t.defined() && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 != 0)
                t = t.clone();
    }
    const NormSizes z(x, w, cos, pos, seq_first);
    const rope_status st = g_norm(address(x[0]), address(x[1]), address(y[0]), address(y[1]), address(w[0]), address(w[1]),
                                  cos.const_data_ptr<float>(), sin.const_data_ptr<float>(),
                                  static_cast<const int32_t *>(address(pos)), z.pos_stride, z.B, z.H[0], z.H[1], z.S, z.D,
                                  z.strides[0], z.strides[1], z.rotary_dim, layout, seq_first, (float)eps, z.code, z.w_code, z.rows,
                                  c10::cuda::getCurrentCUDAStream(cos.get_device()).stream());
    if (st != ROPE_OK || !graph)
        return st;
    const std::shared_ptr<NormRotaryBackward> node(new NormRotaryBackward(), torch::autograd::deleteNode);
    node->set_next_edges(torch::autograd::collect_next_edges(in[0], in[1], in[2], in[3]));
    for (int i = 0; i < 7; ++i) {
        const at::Tensor &t = i < 2 ? x[i] : i < 4 ? w[i - 2] : in[i];
        node->given[i] = t.defined();
        if (t.defined())
            node->saved[i] = torch::autograd::SavedVariable(t, false);
    }
    node->eps = eps;
    node->layout = layout;
    node->seq_first = seq_first;
    for (at::Tensor &t : y)
        if (t.defined())
            torch::autograd::set_history(t, node);
    return ROPE_OK;
}

// Whether a tensor is a leaf whose gradients a graph that is alive accumulates on
// another stream than the current one.  (The engine would make that stream wait for a
// captured backward pass, which ends the capture with an error.)
bool accumulates_elsewhere(const at::Tensor &t)
{
    if (!t.defined() || !t.is_leaf() || !t.requires_grad())
        return false;
    const auto node = torch::autograd::impl::try_get_grad_accumulator(t);
    if (node == nullptr)
        return false;
    const auto stream = node->stream();
    return stream && *stream != c10::cuda::getCurrentCUDAStream(t.get_device()).unwrap();
}

// norm_rotary_qk(q, k, wq, wk, cos, sin, eps, pos_idx, rotary_dim, layout, seq_before_head)
// -> (q_out, k_out), or a status
PyObject *norm_rotary_qk(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 11);
        const bool has_q = a[0] != Py_None, has_k = a[1] != Py_None;
        const at::Tensor &first = has_q ? tensor(a[0], "q") : tensor(a[1], "q or k");
        const Call c(first, Py_None);
        type_code(first, "norm_rotary_qk");
        const at::ScalarType type = first.scalar_type();
        const bool seq_first = truth(a[10]);
        auto given = [&](int i, const char *name) { return a[i] == Py_None ? at::Tensor() : tensor(a[i], name); };
        const at::Tensor q = given(0, "q"), k = given(1, "k"), wq = given(2, "wq"), wk = given(3, "wk"), pos = given(7, "pos_idx");
        // (strides and alignments the library does not take are copied, so features need not be dense)
        struct Shape : Heads {
            Shape(const Call &c, const at::Tensor &t, const char *name, at::ScalarType type, bool seq_first)
                : Heads(c, Py_None, name, type, seq_first)
            {
                if (!t.defined())
                    return;
                c.on_device(t, name, type);
                if (t.dim() != 4)
                    fail(PyExc_ValueError, std::string(name) + " must be 4-dimensional, got " + shape_of(t));
                B = t.size(0);
                S = t.size(seq_first ? 1 : 2);
                if (t.size(seq_first ? 2 : 1) > INT32_MAX || t.size(3) > INT32_MAX)
                    fail(PyExc_ValueError, std::string(name) + " is too large: " + shape_of(t));
                H = (int32_t)t.size(seq_first ? 2 : 1);
                D = (int32_t)t.size(3);
            }
        };
        const Shape qs(c, q, "q", type, seq_first), ks(c, k, "k", type, seq_first);
        const NormShape z(c, qs, ks, has_q, has_k, a[7]);
        const Weight ww(c, a[2], "wq", type, z.D), wv(c, a[3], "wk", type, z.D);
        weight_code(ww, wv, ROPE_F32);
        const Tables t(c, a[4], a[5], a[8]);
        if (t.cos == nullptr || t.sin == nullptr)
            fail(PyExc_ValueError, "cos and sin must have rows");
        const at::Tensor cos = tensor(a[4], "cos"), sin = tensor(a[5], "sin");
        const double eps = number(a[6]);
        const int64_t layout = integer(a[9]);
        const c10::cuda::CUDAGuard guard(c.device);
        for (const at::Tensor &x : {q, k, wq, wk})
            TORCH_CHECK(!x.defined() || !x._fw_grad(0).defined(), "norm_rotary_qk: has no forward-mode derivative");
        if (at::GradMode::is_enabled() &&
            c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) {
            const at::Tensor leaves[4] = {q, k, wq, wk};
            for (int i = 0; i < 4; ++i)
                if (accumulates_elsewhere(leaves[i]))
                    fail(PyExc_RuntimeError, std::string("a graph of ") + (i < 2 ? "" : "w") + (i % 2 ? "k" : "q") +
                                                 " made on another stream is alive: drop it before the backward pass is captured");
        }
        const at::Tensor in[7] = {q, k, wq, wk, cos, sin, pos};
        at::Tensor out[2];
        rope_status st;
        {
            const Unlocked u;
            st = norm_rotary_forward(in, eps, (int32_t)layout, seq_first, out);
        }
        if (st != ROPE_OK)
            return status(st);
        return tuple_of({out[0], out[1]});
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// build_tables_scaled(kind, theta, rotary_dim, rows, pos_offset, factor, original_positions,
//     low_turns, high_turns, value_scale, device (or -1), stream) -> (cos, sin), or a status
PyObject *build_tables_scaled(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 12);
        const int64_t rd = integer(a[2]), rows = integer(a[3]), at = integer(a[10]);
        if (rd < 0 || rd > INT32_MAX || rows < 0)
            return status(ROPE_ERR_INVALID_ARG);
        const c10::DeviceIndex device = at < 0 ? c10::cuda::current_device() : (c10::DeviceIndex)at;
        const Call c(device, a[11]);
        const c10::cuda::CUDAGuard guard(c.device);
        const at::Tensor cos = c.empty_returned({rows, rd / 2}, at::kFloat), sin = c.empty_returned({rows, rd / 2}, at::kFloat);
        const rope_status st = unlocked(g_tables_scaled, (int32_t)integer(a[0]), number(a[1]), (int32_t)rd, rows, integer(a[4]),
                                        number(a[5]), integer(a[6]), number(a[7]), number(a[8]), number(a[9]),
                                        static_cast<float *>(cos.data_ptr()), static_cast<float *>(sin.data_ptr()), c.stream);
        if (st != ROPE_OK)
            return status(st);
        return tuple_of({cos, sin});
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// norm_cache_append(q, k, v, wq, wk, k_pages, v_pages, block_table, cu_seqlens,
//     cache_lens, cos, sin, eps, pos, pos_offset, rotary_dim, layout, q_out, stream)
// -> q_out, or a status
PyObject *norm_cache_append(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    try {
        expect(n, 19);
        const at::Tensor &q = tensor(a[0], "q");
        const Call c(q, a[18]);
        const int32_t code = type16(q, "norm_cache_append");
        const at::ScalarType type = q.scalar_type();
        const Cache pool(c, a[5], a[6], type);
        const Rows qr(c, a[0], "q", type, -1, pool.D), kr(c, a[1], "k", type, pool.Hk, pool.D),
            vr(c, a[2], "v", type, pool.Hk, pool.D);
        if (kr.n != vr.n || kr.n != qr.n)
            fail(PyExc_ValueError, "q, k and v must have the same tokens");
        const Weight wq(c, a[3], "wq", type, pool.D), wk(c, a[4], "wk", type, pool.D);
        const at::Tensor &table = tensor(a[7], "block_table");
        if (table.dim() != 2)
            fail(PyExc_ValueError, "block_table must be [n_seqs, max_blocks], got " + shape_of(table));
        const int64_t seqs = table.size(0), blocks = table.size(1);
        const Tables t(c, a[10], a[11], a[15]);
        const int32_t *list = c.ints(a[7], "block_table", -1), *cu = c.ints(a[8], "cu_seqlens", seqs + 1),
                      *lens = c.ints(a[9], "cache_lens", seqs), *pos = c.ints(a[13], "pos", kr.n, true);
        const c10::cuda::CUDAGuard guard(c.device);
        const at::Tensor out = output(c, a[17], qr, type, "q_out");
        const rope_status st =
            unlocked(g_norm_append, qr.p, kr.p, vr.p, out.data_ptr(), pool.k, pool.v, wq.p, wk.p, list, cu, lens, t.cos, t.sin,
                     pos, integer(a[14]), seqs, kr.n, qr.stride, kr.stride, vr.stride, qr.H, pool.Hk, pool.D, t.rotary_dim,
                     (int32_t)integer(a[16]), (float)number(a[12]), pool.page, pool.n_pages, blocks, code,
                     weight_code(wq, wk, code), t.rows, c.stream);
        if (st != ROPE_OK)
            return status(st);
        written(tensor(a[5], "k_pages"));
        written(tensor(a[6], "v_pages"));
        if (a[17] != Py_None)
            written(out);
        return THPVariable_Wrap(out);
    } catch (const PythonError &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_append)), METH_FASTCALL, nullptr},
    {"attention_packed", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_packed)), METH_FASTCALL,
     nullptr},
    {"attention_shared_prefix", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_shared_prefix)),
     METH_FASTCALL, nullptr},
    {"attention_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_paged)), METH_FASTCALL,
     nullptr},
    {"norm_rotate_qk", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rotate_qk)), METH_FASTCALL, nullptr},
    {"norm_rotate_qk_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rotate_qk_backward)),
     METH_FASTCALL, nullptr},
    {"norm_rotary_qk", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_rotary_qk)), METH_FASTCALL, nullptr},
    {"build_tables_scaled", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(build_tables_scaled)), METH_FASTCALL,
     nullptr},
    {"norm_cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(norm_cache_append)), METH_FASTCALL,
     nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
