// Compiled half of the Python binding for the streaming calls: reads and checks a
// call's tensors and makes the call.
//
// A decode step is a few small calls, and a call read in Python takes 7 us (some fifty
// attribute look-ups) for 8 us of GPU work; read here it takes one.  A function returns
// None for arguments that it does not take (wrong types, shapes, devices, layouts,
// anything that throws): the binding then goes through them in Python, which names what
// is wrong.  It returns an int, the library's status, where the library refuses the
// call.  The library's functions are reached through the addresses that bind() is given,
// so that one library is loaded once.
#include <Python.h>

#include <climits>
#include <cmath>

#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attn_sm103a.h"

namespace {

struct Library {
    decltype(&attn_cache_append) cache_append = nullptr;
    decltype(&attn_fwd_cache_workspace_bytes) fwd_cache_workspace_bytes = nullptr;
    decltype(&attn_fwd_cache) fwd_cache = nullptr;
    decltype(&attn_fwd_sinks) fwd_sinks = nullptr;
    decltype(&attn_bwd_sinks_workspace_bytes) bwd_sinks_workspace_bytes = nullptr;
    decltype(&attn_bwd_sinks) bwd_sinks = nullptr;
} lib;

struct Unread {};  // arguments for the Python half

void need(bool ok) {
    if (!ok) throw Unread();
}

const at::Tensor& tensor(PyObject* o) {
    need(THPVariable_Check(o));
    return THPVariable_Unpack(o);
}

// A tensor of this type, rank and device.
const at::Tensor& tensor(PyObject* o, at::ScalarType type, int rank, int dev) {
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == type && t.dim() == rank && t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev);
    return t;
}

int size(int64_t n) {
    need(n >= 0 && n <= INT_MAX);
    return static_cast<int>(n);
}

long long integer(PyObject* o) {
    need(PyLong_CheckExact(o));
    const long long x = PyLong_AsLongLong(o);
    need(!(x == -1 && PyErr_Occurred()));
    return x;
}
int small(PyObject* o) {
    const long long x = integer(o);
    need(x >= INT_MIN && x <= INT_MAX);
    return static_cast<int>(x);
}

// [B, heads, N, d] (or [B, N, heads, d]) of bf16, d contiguous.
struct Rows {
    const at::Tensor* t;
    int B, H, N, D;
    attn_strides_t st;
    void* p() const { return t->data_ptr(); }
};
Rows rows(PyObject* o, int dev, bool bnhd) {
    Rows r;
    r.t = &tensor(o, at::kBFloat16, 4, dev);
    const auto n = r.t->sizes(), s = r.t->strides();
    need(s[3] == 1);
    const int h = bnhd ? 2 : 1, x = bnhd ? 1 : 2;
    r.B = size(n[0]), r.H = size(n[h]), r.N = size(n[x]), r.D = size(n[3]);
    r.st = {s[0], s[h], s[x]};
    return r;
}
Rows rows_like(PyObject* o, const Rows& like, int dev, bool bnhd) {
    const Rows r = rows(o, dev, bnhd);
    need(r.t->sizes() == like.t->sizes());
    return r;
}

// A contiguous tensor of this shape.
void* dense(PyObject* o, at::ScalarType type, at::IntArrayRef shape, int dev) {
    const at::Tensor& t = tensor(o, type, static_cast<int>(shape.size()), dev);
    need(t.sizes() == shape && t.is_contiguous());
    return t.data_ptr();
}

// So many bytes one after the other (an expanded tensor counts bytes that it does not have).
void* workspace(const at::Tensor& t, size_t room, int dev) {
    need(room > 0 && t.layout() == at::kStrided && t.is_cuda() && t.get_device() == dev && t.nbytes() >= room && t.is_contiguous());
    return t.data_ptr();
}

float scale_of(PyObject* o, int D) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
    need(PyFloat_CheckExact(o));
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
}

attn_cache_t cache_of(PyObject* const* a, int dev, int B, int Hk, int D) {  // k_pages, v_pages, scales, table, lengths
    const at::Tensor& k = tensor(a[0], at::kByte, 4, dev);
    const at::Tensor& v = tensor(a[1], at::kByte, 4, dev);
    const at::Tensor& table = tensor(a[4], at::kInt, 2, dev);
    const auto n = k.sizes(), ks = k.strides(), vs = v.strides();
    need(v.sizes() == n && n[1] == Hk && n[3] == D && ks[3] == 1 && vs[3] == 1);
    need(table.size(0) == B && table.size(1) >= 1 && (table.stride(1) == 1 || table.size(1) == 1));
    attn_cache_t c;
    c.k_pages = k.data_ptr();
    c.v_pages = v.data_ptr();
    c.ks = {ks[0], ks[1], ks[2]};
    c.vs = {vs[0], vs[1], vs[2]};
    c.k_scale = static_cast<float*>(dense(a[2], at::kFloat, {n[0], n[1]}, dev));
    c.v_scale = static_cast<float*>(dense(a[3], at::kFloat, {n[0], n[1]}, dev));
    c.page_table = static_cast<const int32_t*>(table.data_ptr());
    c.table_stride = table.stride(0);
    c.seq_lens = static_cast<const int32_t*>(dense(a[5], at::kInt, {B}, dev));
    c.num_pages = size(n[0]);
    c.page_size = size(n[2]);
    c.max_pages = size(table.size(1));
    return c;
}

const int32_t* lens_or_null(PyObject* o, int B, int dev) {
    return o == Py_None ? nullptr : static_cast<const int32_t*>(dense(o, at::kInt, {B}, dev));
}

// An output that was given, or a new one; holds a reference either way.
struct Out {
    PyObject* o;
    Out(PyObject* given, const at::Tensor* made) : o(given) {
        if (made != nullptr) o = THPVariable_Wrap(*made);
        else Py_INCREF(o);
        need(o != nullptr);
    }
    ~Out() { Py_XDECREF(o); }
    Out(const Out&) = delete;
    PyObject* release() {
        PyObject* r = o;
        o = nullptr;
        return r;
    }
};
Out like_or_given(PyObject* o, const Rows& like) {
    if (o != Py_None) return Out(o, nullptr);
    const at::Tensor t = at::empty_like(*like.t);
    return Out(nullptr, &t);
}
Out lse_or_given(PyObject* o, const Rows& q) {
    if (o != Py_None) return Out(o, nullptr);
    const at::Tensor t = at::empty({q.B, q.H, q.N}, q.t->options().dtype(at::kFloat));
    return Out(nullptr, &t);
}

template <typename F>
attn_status called(F call) {  // without the interpreter's lock: a launch may wait for room in the stream
    PyThreadState* s = PyEval_SaveThread();
    const attn_status rc = call();
    PyEval_RestoreThread(s);
    return rc;
}

template <typename... O>
PyObject* outputs(attn_status rc, O&... o) {
    if (rc != ATTN_OK) return PyLong_FromLong(rc);
    PyObject* t = PyTuple_New(sizeof...(o));
    if (t == nullptr) return nullptr;
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(t, i++, o.release()), ...);
    return t;
}

// Any exception: the Python half goes through the arguments again.
template <typename F>
PyObject* guarded(bool ok, F f) {
    try {
        need(ok);
        return f();
    } catch (...) {
        PyErr_Clear();
        Py_RETURN_NONE;
    }
}

// k, v, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, new_lens, bnhd, dev, stream
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n == 12 && lib.cache_append, [&]() -> PyObject* {
        const bool bnhd = a[9] == Py_True;
        const int dev = small(a[10]);
        const Rows k = rows(a[0], dev, bnhd), v = rows_like(a[1], k, dev, bnhd);
        const attn_cache_t c = cache_of(a + 2, dev, k.B, k.H, k.D);
        const int32_t* lens = lens_or_null(a[8], k.B, dev);
        auto stream = reinterpret_cast<attn_stream_t>(integer(a[11]));
        return PyLong_FromLong(called([&] {
            return lib.cache_append(&c, k.p(), k.st, v.p(), v.st, lens, k.B, k.H, k.N, k.D, stream);
        }));
    });
}

// q, k_pages, v_pages, k_scale, v_scale, page_table, seq_lens, q_lens, bnhd, scale, left, sinks, o, lse, workspace, dev, stream
PyObject* fwd_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n == 17 && lib.fwd_cache, [&]() -> PyObject* {
        const bool bnhd = a[8] == Py_True;
        const int dev = small(a[15]);
        const Rows q = rows(a[0], dev, bnhd);
        const int Hk = size(tensor(a[1], at::kByte, 4, dev).size(1));
        const attn_cache_t c = cache_of(a + 1, dev, q.B, Hk, q.D);
        const int32_t* lens = lens_or_null(a[7], q.B, dev);
        const float scale = scale_of(a[9], q.D);
        const int left = small(a[10]), sinks = small(a[11]);
        const size_t room = lib.fwd_cache_workspace_bytes(q.B, q.H, Hk, q.N, q.D);
        void* w = workspace(tensor(a[14]), room, dev);
        Out o = like_or_given(a[12], q), lse = lse_or_given(a[13], q);
        const Rows ov = rows_like(o.o, q, dev, bnhd);
        float* l = static_cast<float*>(dense(lse.o, at::kFloat, {q.B, q.H, q.N}, dev));
        auto stream = reinterpret_cast<attn_stream_t>(integer(a[16]));
        const attn_status rc = called([&] {
            return lib.fwd_cache(&c, q.p(), q.st, ov.p(), ov.st, l, w, lens, q.B, q.H, Hk, q.N, q.D, scale, left, sinks,
                                 stream);
        });
        return outputs(rc, o, lse);
    });
}

// q, k, v, left, sinks, right, bnhd, scale, o, lse, dev, stream
PyObject* fwd_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n == 12 && lib.fwd_sinks, [&]() -> PyObject* {
        const bool bnhd = a[6] == Py_True;
        const int dev = small(a[10]), left = small(a[3]), sinks = small(a[4]), right = small(a[5]);
        const Rows q = rows(a[0], dev, bnhd), k = rows(a[1], dev, bnhd), v = rows_like(a[2], k, dev, bnhd);
        need(k.B == q.B && k.N == q.N && k.D == q.D);
        const float scale = scale_of(a[7], q.D);
        Out o = like_or_given(a[8], q), lse = lse_or_given(a[9], q);
        const Rows ov = rows_like(o.o, q, dev, bnhd);
        float* l = static_cast<float*>(dense(lse.o, at::kFloat, {q.B, q.H, q.N}, dev));
        auto stream = reinterpret_cast<attn_stream_t>(integer(a[11]));
        const attn_status rc = called([&] {
            return lib.fwd_sinks(q.p(), q.st, k.p(), k.st, v.p(), v.st, ov.p(), ov.st, l, q.B, q.H, k.H, q.N, q.D, scale,
                                 left, right, sinks, stream);
        });
        return outputs(rc, o, lse);
    });
}

// q, k, v, o, dout, lse, left, sinks, right, bnhd, scale, dq, dk, dv, workspace, dev, stream
PyObject* bwd_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n == 17 && lib.bwd_sinks, [&]() -> PyObject* {
        const bool bnhd = a[9] == Py_True;
        const int dev = small(a[15]), left = small(a[6]), sinks = small(a[7]), right = small(a[8]);
        const Rows q = rows(a[0], dev, bnhd), k = rows(a[1], dev, bnhd), v = rows_like(a[2], k, dev, bnhd);
        need(k.B == q.B && k.N == q.N && k.D == q.D);
        const Rows o = rows_like(a[3], q, dev, bnhd), dout = rows_like(a[4], q, dev, bnhd);
        const float* l = static_cast<float*>(dense(a[5], at::kFloat, {q.B, q.H, q.N}, dev));
        const float scale = scale_of(a[10], q.D);
        const size_t room = lib.bwd_sinks_workspace_bytes(q.B, q.H, k.H, q.N, q.D, sinks);
        need(room > 0);
        Out dq = like_or_given(a[11], q), dk = like_or_given(a[12], k), dv = like_or_given(a[13], v);
        const Rows dqv = rows_like(dq.o, q, dev, bnhd), dkv = rows_like(dk.o, k, dev, bnhd), dvv = rows_like(dv.o, v, dev, bnhd);
        const at::Tensor ws = a[14] != Py_None ? tensor(a[14])
                                               : at::empty({static_cast<int64_t>(room)}, q.t->options().dtype(at::kByte));
        void* w = workspace(ws, room, dev);
        auto stream = reinterpret_cast<attn_stream_t>(integer(a[16]));
        const attn_status rc = called([&] {
            return lib.bwd_sinks(q.p(), q.st, k.p(), k.st, v.p(), v.st, o.p(), o.st, dout.p(), dout.st, l, dqv.p(), dqv.st,
                                 dkv.p(), dkv.st, dvv.p(), dvv.st, w, q.B, q.H, k.H, q.N, q.D, scale, left, right, sinks,
                                 stream);
        });
        return outputs(rc, dq, dk, dv);
    });
}

// Addresses of the library's functions, in the order of Library.
PyObject* bind(PyObject*, PyObject* args) {
    unsigned long long p[6];
    if (!PyArg_ParseTuple(args, "KKKKKK", p, p + 1, p + 2, p + 3, p + 4, p + 5)) return nullptr;
    lib.cache_append = reinterpret_cast<decltype(lib.cache_append)>(p[0]);
    lib.fwd_cache_workspace_bytes = reinterpret_cast<decltype(lib.fwd_cache_workspace_bytes)>(p[1]);
    lib.fwd_cache = reinterpret_cast<decltype(lib.fwd_cache)>(p[2]);
    lib.fwd_sinks = reinterpret_cast<decltype(lib.fwd_sinks)>(p[3]);
    lib.bwd_sinks_workspace_bytes = reinterpret_cast<decltype(lib.bwd_sinks_workspace_bytes)>(p[4]);
    lib.bwd_sinks = reinterpret_cast<decltype(lib.bwd_sinks)>(p[5]);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)); }

PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"cache_append", fast(cache_append), METH_FASTCALL, nullptr},
                         {"fwd_cache", fast(fwd_cache), METH_FASTCALL, nullptr},
                         {"fwd_sinks", fast(fwd_sinks), METH_FASTCALL, nullptr},
                         {"bwd_sinks", fast(bwd_sinks), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the PyTorch and Python whose headers this was compiled with (set by the build),
// which the binding compares with those that it runs in.
PyMODINIT_FUNC PyInit__attn_call() {
    PyObject* m = PyModule_Create(&module);
    if (m != nullptr && PyModule_AddStringConstant(m, "built_for", ATTN_BUILT_FOR) != 0) Py_CLEAR(m);
    return m;
}
