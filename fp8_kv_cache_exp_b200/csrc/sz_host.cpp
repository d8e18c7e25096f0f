// sz_host.cpp -- the Python binding's argument checks of the operators on a paged
// cache, as a CPython module: tensors to the argument structs of
// include/splitzip.h, and the call.
//
// Decoding calls these operators once per layer and token, with a dozen tensors
// each; in Python the checks and the packing of one call took 6 to 7 us, twice
// what the rest of the call and the kernel take.  The module links to torch for
// its tensors' fields only; libsplitzip's entry points are handed in by address
// (bind), so that there is one copy of the library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "splitzip.h"

namespace {

using AppendFn = sz_status (*)(const sz_kv_cache_t *, const sz_kv_append_t *, void *, size_t, cudaStream_t);
using NormRopeFn = sz_status (*)(const sz_qk_norm_rope_t *, void *, size_t, cudaStream_t);
using AttnFn = sz_status (*)(const sz_kv_cache_t *, const sz_attn_t *, void *, size_t, cudaStream_t);
AppendFn g_append;
NormRopeFn g_norm_rope;
AttnFn g_attn;

// A refused argument: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(PyObject *kind, const char *format, const char *name, long n = 0) {
    PyErr_Format(kind, format, name, n);
    throw Refused{};
}

const at::Tensor *tensor(PyObject *o, const char *name, bool optional = false) {
    if (o == Py_None && optional) return nullptr;
    if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s: a tensor", name);
    return &THPVariable_Unpack(o);
}

// The device that all of a call's tensors are on, which is the current one.
struct Device {
    int64_t index;
    void add(const at::Tensor *t) const {
        if (t && (t->is_cuda() ? int64_t(t->get_device()) : -1) != index) {
            PyErr_SetString(PyExc_ValueError, "all tensors must be on the cache's device (the first tensor's)");
            throw Refused{};
        }
    }
    void check() const {
        if (index < 0 || int64_t(c10::cuda::current_device()) != index) {
            PyErr_SetString(PyExc_ValueError, "the tensors' CUDA device must be the current device");
            throw Refused{};
        }
    }
};

int64_t device_of(const at::Tensor *t) { return t->is_cuda() ? int64_t(t->get_device()) : -1; }

// A bfloat16 view [tokens, heads, dim] whose rows are contiguous.
sz_heads_t heads(const at::Tensor *t, int64_t dim, int64_t tokens, const char *name) {
    if (t->scalar_type() != at::kBFloat16) refuse(PyExc_TypeError, "%s: bfloat16", name);
    if (t->dim() != 3 || t->size(2) != dim) refuse(PyExc_ValueError, "%s: [tokens, heads, %ld]", name, long(dim));
    if (t->size(0) != tokens) refuse(PyExc_ValueError, "%s: must have %ld tokens", name, long(tokens));
    if (t->stride(2) != 1) refuse(PyExc_ValueError, "%s: a head's elements must be contiguous", name);
    sz_heads_t h{};
    h.data = t->data_ptr();
    h.token_stride = tokens > 1 ? uint64_t(t->stride(0)) : 0;
    h.head_stride = t->size(1) > 1 ? uint64_t(t->stride(1)) : 0;
    h.heads = uint32_t(t->size(1));
    return h;
}

// Data of a contiguous vector of n elements (null for none).
template <typename T>
T *vector(const at::Tensor *t, at::ScalarType type, int64_t n, const char *name) {
    if (!t) return nullptr;
    if (t->scalar_type() != type) {
        const char *want = type == at::kInt ? "%s: torch.int32" : type == at::kFloat ? "%s: torch.float32" : "%s: torch.bfloat16";
        refuse(PyExc_TypeError, want, name);
    }
    if (t->numel() != n || !t->is_contiguous()) refuse(PyExc_ValueError, "%s: %ld contiguous elements", name, long(n));
    return static_cast<T *>(t->data_ptr());
}

void *workspace(const at::Tensor *t, size_t *bytes) {
    if (!t->is_contiguous()) {
        PyErr_SetString(PyExc_ValueError, "the workspace must be contiguous");
        throw Refused{};
    }
    *bytes = size_t(t->nbytes());
    return t->data_ptr();
}

double number(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refused{};
    return x;
}

int64_t whole(PyObject *o, const char *name, int64_t most) {
    const long long x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused{};
    if (x < 0 || x > most) refuse(PyExc_ValueError, "%s: 0 to %ld", name, long(most));
    return x;
}

bool truth(PyObject *o) {
    const int x = PyObject_IsTrue(o);
    if (x < 0) throw Refused{};
    return x != 0;
}

// A raw stream address, or None for the device's current stream.
cudaStream_t stream(PyObject *o, int64_t device) {
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(device)).stream();
    void *s = PyLong_AsVoidPtr(o);
    if (!s && PyErr_Occurred()) throw Refused{};
    return static_cast<cudaStream_t>(s);
}

const sz_kv_cache_t *cache_struct(PyObject *o) {
    if (!PyBytes_Check(o) || PyBytes_GET_SIZE(o) != Py_ssize_t(sizeof(sz_kv_cache_t))) {
        PyErr_SetString(PyExc_TypeError, "cache: a KVCache");
        throw Refused{};
    }
    return reinterpret_cast<const sz_kv_cache_t *>(PyBytes_AS_STRING(o));
}

struct NormRope {
    const at::Tensor *q_norm, *k_norm, *rope, *positions;
    void fill(sz_head_norm_t &n, sz_rope_t &r, int64_t dim, int64_t tokens, PyObject *eps, PyObject *interleaved) const {
        n.q_weight = vector<void>(q_norm, at::kBFloat16, dim, "q_norm");
        n.k_weight = vector<void>(k_norm, at::kBFloat16, dim, "k_norm");
        n.eps = float(number(eps));
        if (!rope) return;
        if (rope->dim() != 2) refuse(PyExc_ValueError, "%s: [positions, rot]", "rope");
        if (rope->size(0) > 0x7fffffff || rope->size(1) > 256) refuse(PyExc_ValueError, "%s: too large", "rope");
        r.table = vector<const float>(rope, at::kFloat, rope->numel(), "rope");
        r.positions = vector<const int32_t>(positions, at::kInt, tokens, "positions");
        r.table_len = uint32_t(rope->size(0));
        r.rot = uint32_t(rope->size(1));
        r.interleaved = truth(interleaved);
    }
};

// The library's call, which waits while the stream's queue of launches is full:
// other Python threads run meanwhile, as in a call through ctypes.  (The caller
// holds its tensors and the cache's struct.)
template <typename F, typename... Args>
sz_status unlocked(F call, Args... args) {
    PyThreadState *state = PyEval_SaveThread();
    const sz_status s = call(args...);
    PyEval_RestoreThread(state);
    return s;
}

template <typename F>
PyObject *guarded(Py_ssize_t have, Py_ssize_t want, F &&f) {
    if (have != want) {
        PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
        return nullptr;
    }
    try {
        return PyLong_FromLong(long(f()));
    } catch (const Refused &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// append(cache, device, k, v, cu_q, kv_len, ws, q, q_out, q_norm, k_norm, eps, rope, positions, interleaved, stream)
PyObject *append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 16, [&] {
        const sz_kv_cache_t *c = cache_struct(a[0]);
        const Device dev{PyLong_AsLongLong(a[1])};
        const at::Tensor *k = tensor(a[2], "k"), *v = tensor(a[3], "v"), *cu_q = tensor(a[4], "cu_q"),
                         *kv_len = tensor(a[5], "kv_len"), *ws = tensor(a[6], "ws"), *q = tensor(a[7], "q", true),
                         *q_out = tensor(a[8], "q_out", true);
        const NormRope nr{tensor(a[9], "q_norm", true), tensor(a[10], "k_norm", true), tensor(a[12], "rope", true),
                          tensor(a[13], "positions", true)};
        for (const at::Tensor *t : {k, v, cu_q, kv_len, ws, q, q_out, nr.q_norm, nr.k_norm, nr.rope, nr.positions}) dev.add(t);
        dev.check();
        if (q_out && !q) refuse(PyExc_ValueError, "%s without q", "q_out");
        const int64_t dim = c->head_dim, tokens = k->dim() > 0 ? k->size(0) : 0;
        sz_kv_append_t s{};
        s.tokens = uint64_t(tokens);
        s.k = heads(k, dim, tokens, "k");
        s.v = heads(v, dim, tokens, "v");
        if (q) {
            s.q = heads(q, dim, tokens, "q");
            s.q_out = q_out ? heads(q_out, dim, tokens, "q_out") : s.q;
        }
        s.cu_q = vector<const int32_t>(cu_q, at::kInt, int64_t(c->seqs) + 1, "cu_q");
        s.kv_len = vector<const int32_t>(kv_len, at::kInt, c->seqs, "kv_len");
        nr.fill(s.norm, s.rope, dim, tokens, a[11], a[14]);
        size_t bytes;
        void *w = workspace(ws, &bytes);
        return unlocked(g_append, c, &s, w, bytes, stream(a[15], dev.index));
    });
}

// norm_rope(q, k, q_out, k_out, ws, q_norm, k_norm, eps, rope, positions, interleaved, stream)
PyObject *norm_rope(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const at::Tensor *q = tensor(a[0], "q", true), *k = tensor(a[1], "k", true), *q_out = tensor(a[2], "q_out", true),
                         *k_out = tensor(a[3], "k_out", true), *ws = tensor(a[4], "ws");
        const NormRope nr{tensor(a[5], "q_norm", true), tensor(a[6], "k_norm", true), tensor(a[8], "rope", true),
                          tensor(a[9], "positions", true)};
        const at::Tensor *x = q ? q : k;
        if (!x) refuse(PyExc_ValueError, "%s or k", "q");
        const Device dev{device_of(x)};
        for (const at::Tensor *t : {q, k, q_out, k_out, ws, nr.q_norm, nr.k_norm, nr.rope, nr.positions}) dev.add(t);
        dev.check();
        if (!q != !q_out) refuse(PyExc_ValueError, "%s and q_out come together", "q");
        if (!k != !k_out) refuse(PyExc_ValueError, "%s and k_out come together", "k");
        if (x->dim() != 3) refuse(PyExc_ValueError, "%s: [tokens, heads, head_dim]", q ? "q" : "k");
        const int64_t dim = x->size(2), tokens = x->size(0);
        if (dim > 256) refuse(PyExc_ValueError, "%s: heads of at most 256 elements", q ? "q" : "k");
        sz_qk_norm_rope_t s{};
        s.tokens = uint64_t(tokens);
        if (q) s.q = heads(q, dim, tokens, "q"), s.q_out = heads(q_out, dim, tokens, "q_out");
        if (k) s.k = heads(k, dim, tokens, "k"), s.k_out = heads(k_out, dim, tokens, "k_out");
        nr.fill(s.norm, s.rope, dim, tokens, a[7], a[10]);
        s.head_dim = uint32_t(dim);
        size_t bytes;
        void *w = workspace(ws, &bytes);
        return unlocked(g_norm_rope, &s, w, bytes, stream(a[11], dev.index));
    });
}

// attn(cache, device, q, cu_q, kv_len, out, ws, scale, causal, window, lse, stream)
PyObject *attn(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 12, [&] {
        const sz_kv_cache_t *c = cache_struct(a[0]);
        const Device dev{PyLong_AsLongLong(a[1])};
        const at::Tensor *q = tensor(a[2], "q"), *cu_q = tensor(a[3], "cu_q"), *kv_len = tensor(a[4], "kv_len"),
                         *out = tensor(a[5], "out"), *ws = tensor(a[6], "ws"), *lse = tensor(a[10], "lse", true);
        for (const at::Tensor *t : {q, cu_q, kv_len, out, ws, lse}) dev.add(t);
        dev.check();
        const int64_t dim = c->head_dim, tokens = q->dim() > 0 ? q->size(0) : 0;
        sz_attn_t s{};
        s.tokens = uint64_t(tokens);
        s.q = heads(q, dim, tokens, "q");
        s.out = heads(out, dim, tokens, "out");
        s.cu_q = vector<const int32_t>(cu_q, at::kInt, int64_t(c->seqs) + 1, "cu_q");
        s.kv_len = vector<const int32_t>(kv_len, at::kInt, c->seqs, "kv_len");
        s.lse = vector<float>(lse, at::kFloat, tokens * s.q.heads, "lse");
        s.scale = float(number(a[7]));
        s.causal = truth(a[8]);
        s.window = uint32_t(whole(a[9], "window", 0x7fffffff));
        size_t bytes;
        void *w = workspace(ws, &bytes);
        return unlocked(g_attn, c, &s, w, bytes, stream(a[11], dev.index));
    });
}

// bind(append, norm_rope, attn): addresses of libsplitzip's entry points
PyObject *bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded(n, 3, [&] {
        g_append = reinterpret_cast<AppendFn>(PyLong_AsVoidPtr(a[0]));
        g_norm_rope = reinterpret_cast<NormRopeFn>(PyLong_AsVoidPtr(a[1]));
        g_attn = reinterpret_cast<AttnFn>(PyLong_AsVoidPtr(a[2]));
        return g_append && g_norm_rope && g_attn ? 0 : 1;
    });
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(bind)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(append)), METH_FASTCALL, nullptr},
    {"norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_rope)), METH_FASTCALL, nullptr},
    {"attn", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(attn)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_host", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__host() { return PyModule_Create(&kModule); }
