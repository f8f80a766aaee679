// serving_binding.cpp -- the Python side of the serving calls: checks of tensors,
// allocation of outputs and workspaces, and the call into librope.
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
#include <string>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "rope.h"

namespace {

decltype(&rope_cache_append) g_append = nullptr;
decltype(&rope_attention_packed_fwd) g_packed = nullptr;
decltype(&rope_attention_packed_workspace) g_packed_bytes = nullptr;
decltype(&rope_attention_decode_fwd) g_decode = nullptr;
decltype(&rope_attention_decode_workspace) g_decode_bytes = nullptr;

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

    Call(const at::Tensor &first, PyObject *s)
    {
        if (!first.is_cuda())
            fail(PyExc_ValueError, "expected CUDA tensors, got one on " + first.device().str());
        device = first.get_device();
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
at::Tensor output(const Call &c, PyObject *given, const Rows &like, at::ScalarType type)
{
    if (given == Py_None)
        return c.empty_returned({like.n, like.H, like.D}, type);
    const at::Tensor &t = tensor(given, "out");
    c.dense(given, "out", type, -1);
    if (t.dim() != 3 || t.size(0) != like.n || t.size(1) != like.H || t.size(2) != like.D)
        fail(PyExc_ValueError, "out must be [" + std::to_string(like.n) + ", " + std::to_string(like.H) + ", " +
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

// bind(addresses of the five entry points)
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    if (n != 5) {
        PyErr_SetString(PyExc_TypeError, "expected 5 addresses");
        return nullptr;
    }
    void *p[5];
    for (int i = 0; i < 5; ++i) {
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

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"cache_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(cache_append)), METH_FASTCALL, nullptr},
    {"attention_packed", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_packed)), METH_FASTCALL,
     nullptr},
    {"attention_shared_prefix", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention_shared_prefix)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
