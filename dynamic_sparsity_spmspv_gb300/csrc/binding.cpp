// Python binding of the decoding step's operators: checks tensors, allocates
// what is returned and calls the C ABI, without going through Python objects
// for every size and address (a call of this kind costs a few microseconds on
// the host, as much as the smallest kernels take).
#include <Python.h>

#include <cmath>
#include <string>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/dbspmspv.h"

namespace {

PyObject *g_error = nullptr;          // DbsError(function, status, why)

struct Failed {};                     // a Python exception is set

[[noreturn]] void fail(const char *fn, int status, const std::string &why)
{
    if (PyObject *e = g_error ? PyObject_CallFunction(g_error, "sis", fn, status, why.c_str()) : nullptr) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, why.c_str());
    }
    throw Failed();
}

[[noreturn]] void bad(const char *fn, const std::string &why) { fail(fn, DBS_ERR_INVALID_ARG, why); }

void check(const char *fn, dbs_status st)
{
    if (st != DBS_OK) fail(fn, st, "");
}

// The arguments of a call by position or name; absent ones are NULL.
template <int N>
struct Args {
    PyObject *v[N] = {};
    Args(const char *fn, PyObject *const (&names)[N], int positional, int required, PyObject *const *args, Py_ssize_t nargs,
         PyObject *kw)
    {
        if (nargs > positional) {
            PyErr_Format(PyExc_TypeError, "%s takes at most %d positional arguments", fn, positional);
            throw Failed();
        }
        for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
        const Py_ssize_t nkw = kw ? PyTuple_GET_SIZE(kw) : 0;
        for (Py_ssize_t k = 0; k < nkw; ++k) {
            PyObject *name = PyTuple_GET_ITEM(kw, k);
            int at = -1;
            for (int i = 0; i < N && at < 0; ++i)
                if (names[i] == name) at = i;
            for (int i = 0; i < N && at < 0; ++i)
                if (PyUnicode_Compare(names[i], name) == 0) at = i;
            if (at < 0 || v[at]) {
                PyErr_Format(PyExc_TypeError, "%s: argument %R is unknown or given twice", fn, name);
                throw Failed();
            }
            v[at] = args[nargs + k];
        }
        for (int i = 0; i < N; ++i) {
            if (!v[i] && i < required) {
                PyErr_Format(PyExc_TypeError, "%s: argument %R is missing", fn, names[i]);
                throw Failed();
            }
            if (v[i] == Py_None) v[i] = nullptr;
        }
    }
};

template <int N>
struct Names {
    PyObject *v[N];
    explicit Names(const char *const (&n)[N])
    {
        for (int i = 0; i < N; ++i) v[i] = PyUnicode_InternFromString(n[i]);
    }
};

bool truth(PyObject *o, bool otherwise)
{
    if (!o) return otherwise;
    const int t = PyObject_IsTrue(o);
    if (t < 0) throw Failed();
    return t != 0;
}

int64_t whole(PyObject *o, int64_t otherwise)
{
    if (!o) return otherwise;
    PyObject *i = PyNumber_Index(o);
    if (!i) throw Failed();
    const long long v = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred()) throw Failed();
    return v;
}

double real(PyObject *o, double otherwise)
{
    if (!o) return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Failed();
    return v;
}

// One call: its name, its device (that of its first tensor, the current one)
// and its stream.
struct Call {
    const char *fn;
    int dev = -1;
    cudaStream_t stream = nullptr;
    bool here = true;                 // the stream is the current one

    // NULL where the argument is absent
    const at::Tensor *tensor(const char *name, PyObject *o)
    {
        if (!o) return nullptr;
        if (!THPVariable_Check(o)) bad(fn, std::string(name) + " has to be a CUDA tensor");
        const at::Tensor &t = THPVariable_Unpack(o);
        if (!t.is_cuda()) bad(fn, std::string(name) + " has to be a CUDA tensor");
        if (t.requires_grad() && at::GradMode::is_enabled())
            bad(fn, std::string(name) + " requires a gradient, and nothing is recorded for autograd: detach it, or call under torch.no_grad()");
        const int d = t.get_device();
        if (dev < 0) {
            dev = d;
            if (d != c10::cuda::current_device()) bad(fn, "tensors have to be on the current CUDA device");
        } else if (d != dev) {
            bad(fn, std::string(name) + " has to be on the same CUDA device");
        }
        return &t;
    }
    const at::Tensor &need(const char *name, PyObject *o)
    {
        const at::Tensor *t = tensor(name, o);
        if (!t) bad(fn, std::string(name) + " has to be a CUDA tensor");
        return *t;
    }
    void on(PyObject *s)
    {
        const cudaStream_t current = c10::cuda::getCurrentCUDAStream(dev).stream();
        stream = current;
        if (!s) return;
        PyObject *h = PyObject_GetAttrString(s, "cuda_stream");
        if (!h) {
            PyErr_Clear();
            h = PyNumber_Index(s);
            if (!h) throw Failed();
        }
        stream = (cudaStream_t)PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!stream && PyErr_Occurred()) throw Failed();
        here = stream == current;
    }
    // Uninitialised, belonging to the call's stream.
    at::Tensor empty(at::IntArrayRef shape, at::ScalarType type)
    {
        const auto o = at::TensorOptions().dtype(type).device(at::Device(at::kCUDA, (c10::DeviceIndex)dev));
        if (here) return at::empty(shape, o);
        const c10::cuda::CUDAStreamGuard guard(stream ? c10::cuda::getStreamFromExternal(stream, (c10::DeviceIndex)dev)
                                                      : c10::cuda::getDefaultCUDAStream((c10::DeviceIndex)dev));
        return at::empty(shape, o);
    }
    dbs_dtype type(const char *name, const at::Tensor &t)
    {
        switch (t.scalar_type()) {
        case at::kFloat: return DBS_F32;
        case at::kHalf: return DBS_F16;
        case at::kBFloat16: return DBS_BF16;
        default: bad(fn, std::string(name) + " has to be float32, float16 or bfloat16");
        }
    }
    // Row stride of a [rows, columns] tensor of that type, rows contiguous.
    int64_t rows(const char *name, const at::Tensor &t, int64_t r, int64_t c, at::ScalarType type)
    {
        if (t.scalar_type() != type || t.dim() != 2 || t.size(0) != r || t.size(1) != c)
            bad(fn, std::string(name) + " has to be " + c10::toString(type) + " [" + std::to_string(r) + ", " + std::to_string(c) + "]");
        if (c > 1 && t.stride(1) != 1) bad(fn, std::string(name) + ": the last dimension has to be contiguous");
        return t.stride(0);
    }
    const void *vector(const char *name, const at::Tensor *t, int64_t n, at::ScalarType type)
    {
        if (!t) return nullptr;
        if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || (n > 1 && t->stride(0) != 1))
            bad(fn, std::string(name) + " has to be contiguous " + c10::toString(type) + " [" + std::to_string(n) + "]");
        return t->data_ptr();
    }
};

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

// A tensor of the caller's that the call writes: autograd has to know if it was saved for a gradient.
void written(const at::Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// Runs a binding's body; a C++ exception becomes a Python one.
template <class F>
PyObject *guarded(F f)
{
    try {
        return f();
    } catch (const Failed &) {
        return nullptr;
    } catch (const std::bad_alloc &) {
        return PyErr_NoMemory();
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *t = PyImport_ImportModule("torch"), *oom = t ? PyObject_GetAttrString(t, "OutOfMemoryError") : nullptr;
        if (oom) PyErr_SetString(oom, e.what_without_backtrace());
        Py_XDECREF(oom);
        Py_XDECREF(t);
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// ---- 4-bit linear layers ----

PyObject *w4_linear(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<7> N({"x", "q", "scales", "zeros", "group", "y", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_w4_linear"};
        const Args<7> a(c.fn, N.v, 4, 3, args, nargs, kw);
        const at::Tensor &x = c.need("x", a.v[0]), &q = c.need("q", a.v[1]), &s = c.need("scales", a.v[2]);
        const at::Tensor *z = c.tensor("zeros", a.v[3]), *given = c.tensor("y", a.v[5]);
        const int64_t group = whole(a.v[4], 128);
        const bool one = x.dim() == 1;
        if ((!one && x.dim() != 2) || q.dim() != 2) bad(c.fn, "x is [tokens, n] or [n], q has two dimensions");
        const int64_t tokens = one ? 1 : x.size(0), n = x.size(-1), m = q.size(0);
        const dbs_dtype dt = c.type("x", x), sd = c.type("scales", s);
        if (group != 32 && group != 64 && group != 128 && group != 256) bad(c.fn, "group has to be 32, 64, 128 or 256");
        if (n > 1 && x.stride(-1) != 1) bad(c.fn, "x: the last dimension has to be contiguous");
        const int64_t groups = (n + group - 1) / group;
        const int64_t qs = c.rows("q", q, m, (n + 1) / 2, at::kByte);
        const int64_t ss = c.rows("scales", s, m, groups, s.scalar_type());
        const int64_t zs = z ? c.rows("zeros", *z, m, groups, at::kByte) : 0;
        c.on(a.v[6]);
        at::Tensor y;
        int64_t ys = m;
        if (given) {
            y = *given;
            if (one && y.dim() == 1) {
                if (y.scalar_type() != x.scalar_type() || y.size(0) != m || (m > 1 && y.stride(0) != 1))
                    bad(c.fn, "y has to be contiguous, in x's type, with a value for each row of q");
            } else {
                ys = c.rows("y", y, tokens, m, x.scalar_type());
            }
        } else {
            y = one ? c.empty({m}, x.scalar_type()) : c.empty({tokens, m}, x.scalar_type());
        }
        check(c.fn, dbs_w4_linear(x.data_ptr(), dt, tokens, one ? n : x.stride(0), (const uint8_t *)q.data_ptr(), qs, s.data_ptr(), sd,
                                  ss, z ? (const uint8_t *)z->data_ptr() : nullptr, zs, m, n, (int32_t)group, y.data_ptr(), ys,
                                  c.stream));
        if (given) written(y);
        return wrap(y);
    });
}

// ---- rotary positions ----

PyObject *rotary_table(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<10> N({"positions", "dim", "base", "scaling", "factor", "trained", "beta_fast", "beta_slow", "device", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_rotary_table"};
        const Args<10> a(c.fn, N.v, 2, 2, args, nargs, kw);
        const int64_t positions = whole(a.v[0], 0), dim = whole(a.v[1], 0);
        int scaling = 0;
        if (a.v[3]) {
            const char *k = PyUnicode_Check(a.v[3]) ? PyUnicode_AsUTF8(a.v[3]) : nullptr;
            const std::string s = k ? k : "";
            scaling = s == "linear" ? DBS_ROTARY_LINEAR : s == "ntk" ? DBS_ROTARY_NTK : s == "yarn" ? DBS_ROTARY_YARN : -1;
            if (scaling < 0) bad(c.fn, "scaling is None, 'linear', 'ntk' or 'yarn'");
        }
        if (positions < 0 || dim < 2 || dim > 512 || dim % 2) bad(c.fn, "positions >= 0, dim even and in 2..512");
        c.dev = c10::cuda::current_device();
        if (a.v[8]) {
            PyObject *s = PyObject_Str(a.v[8]);
            if (!s) throw Failed();
            const char *k = PyUnicode_AsUTF8(s);
            const std::string name = k ? k : "";
            Py_DECREF(s);
            if (name != "cuda" && name != "cuda:" + std::to_string(c.dev)) bad(c.fn, "device has to be the current CUDA device");
        }
        c.on(a.v[9]);
        const at::Tensor t = c.empty({positions, dim}, at::kFloat);
        check(c.fn, dbs_rotary_table(positions, (int32_t)dim, real(a.v[2], 10000.0), (dbs_rotary_scaling)scaling, real(a.v[4], 1.0),
                                     real(a.v[5], 0.0), real(a.v[6], 32.0), real(a.v[7], 1.0), t.data_ptr<float>(), c.stream));
        return wrap(t);
    });
}

// [batch, tokens, heads, head_dim], or without batch.
struct Heads {
    int64_t b, n, h, d, sb, sn, sh;
};

Heads heads_of(const Call &c, const char *name, const at::Tensor &t, at::ScalarType type)
{
    const int64_t k = t.dim();
    if (t.scalar_type() != type || (k != 3 && k != 4))
        bad(c.fn, std::string(name) + " has to be a " + c10::toString(type) + " tensor [batch, tokens, heads, head_dim] or [tokens, heads, head_dim]");
    const Heads H{k == 4 ? t.size(0) : 1, t.size(k - 3), t.size(k - 2), t.size(k - 1), k == 4 ? t.stride(0) : 0,
                  t.stride(k - 3), t.stride(k - 2)};
    if (H.d > 1 && t.stride(k - 1) != 1) bad(c.fn, std::string(name) + ": the last dimension has to be contiguous");
    return H;
}

Heads like(const Call &c, const char *name, const at::Tensor &t, const at::Tensor &q, const Heads &Q)
{
    const Heads H = heads_of(c, name, t, q.scalar_type());
    if (H.b != Q.b || H.n != Q.n || H.d != Q.d) bad(c.fn, std::string(name) + " has to have q's tokens and head size");
    return H;
}

// Checks what every rotation needs; returns q's sizes.
Heads turning(Call &c, const at::Tensor &q, const at::Tensor &table, const at::Tensor &positions, const at::Tensor *slots)
{
    const Heads Q = heads_of(c, "q", q, q.scalar_type());
    if (table.scalar_type() != at::kFloat || table.dim() != 2 || !table.is_contiguous() || table.size(1) > Q.d)
        bad(c.fn, "table has to be contiguous float32 [positions, dim], dim at most head_dim");
    for (const at::Tensor *t : {&positions, slots})
        if (t && (t->scalar_type() != at::kInt || t->numel() != Q.b * Q.n || !t->is_contiguous()))
            bad(c.fn, "positions and slots have to be contiguous int32, one for each token");
    return Q;
}

dbs_rotary_heads part(const at::Tensor &in, const Heads &I, void *out, const Heads &O, bool rotate, bool slots)
{
    return {in.data_ptr(), out, I.sb, I.sn, I.sh, O.sb, O.sn, O.sh, (int32_t)I.h, rotate, slots};
}

// The output for t: `given`, or a new one.
at::Tensor turned(Call &c, const at::Tensor &t, const at::Tensor *given)
{
    if (!given) return c.empty(t.sizes(), t.scalar_type());
    if (given->sizes() != t.sizes()) bad(c.fn, "outputs have their input's shape");
    return *given;
}

PyObject *rotary(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<9> N({"q", "k", "table", "positions", "interleaved", "transposed", "q_out", "k_out", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_rotary"};
        const Args<9> a(c.fn, N.v, 4, 4, args, nargs, kw);
        const at::Tensor &q = c.need("q", a.v[0]), &table = c.need("table", a.v[2]), &pos = c.need("positions", a.v[3]);
        const at::Tensor *k = c.tensor("k", a.v[1]), *qg = c.tensor("q_out", a.v[6]), *kg = c.tensor("k_out", a.v[7]);
        const dbs_dtype dt = c.type("q", q);
        const Heads Q = turning(c, q, table, pos, nullptr);
        const Heads K = k ? like(c, "k", *k, q, Q) : Q;
        c.on(a.v[8]);
        const at::Tensor qo = turned(c, q, qg), ko = k ? turned(c, *k, kg) : at::Tensor();
        dbs_rotary_heads parts[2] = {part(q, Q, qo.data_ptr(), heads_of(c, "q_out", qo, q.scalar_type()), true, false)};
        if (k) parts[1] = part(*k, K, ko.data_ptr(), heads_of(c, "k_out", ko, q.scalar_type()), true, false);
        check(c.fn, dbs_rotary(parts, k ? 2 : 1, dt, Q.b, Q.n, (int32_t)Q.d, (int32_t)table.size(1), table.data_ptr<float>(),
                               table.size(0), pos.data_ptr<int32_t>(), nullptr, 0, 1, truth(a.v[4], false), truth(a.v[5], false),
                               c.stream));
        if (qg) written(qo);
        if (k && kg) written(ko);
        PyObject *r = PyTuple_New(2);
        if (!r) throw Failed();
        PyTuple_SET_ITEM(r, 0, wrap(qo));
        PyTuple_SET_ITEM(r, 1, k ? wrap(ko) : Py_NewRef(Py_None));
        return r;
    });
}

PyObject *rotary_append(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<11> N({"q", "k", "v", "table", "positions", "k_cache", "v_cache", "slots", "interleaved", "q_out", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_rotary_append"};
        const Args<11> a(c.fn, N.v, 8, 8, args, nargs, kw);
        const at::Tensor &q = c.need("q", a.v[0]), &k = c.need("k", a.v[1]), &v = c.need("v", a.v[2]);
        const at::Tensor &table = c.need("table", a.v[3]), &pos = c.need("positions", a.v[4]);
        const at::Tensor &kc = c.need("k_cache", a.v[5]), &vc = c.need("v_cache", a.v[6]), &slots = c.need("slots", a.v[7]);
        const at::Tensor *qg = c.tensor("q_out", a.v[9]);
        const dbs_dtype dt = c.type("q", q);
        const Heads Q = turning(c, q, table, pos, &slots), K = like(c, "k", k, q, Q), V = like(c, "v", v, q, Q);
        if (kc.dim() != 4 || vc.sizes() != kc.sizes() || K.h != V.h)
            bad(c.fn, "caches have to be [pages, page_size, kv_heads, head_dim]");
        const Heads KC = heads_of(c, "k_cache", kc, q.scalar_type()), VC = heads_of(c, "v_cache", vc, q.scalar_type());
        if (KC.h != K.h || KC.d != Q.d) bad(c.fn, "caches have to have k's heads");
        c.on(a.v[10]);
        const at::Tensor qo = turned(c, q, qg);
        const dbs_rotary_heads parts[3] = {part(q, Q, qo.data_ptr(), heads_of(c, "q_out", qo, q.scalar_type()), true, false),
                                           part(k, K, kc.data_ptr(), KC, true, true), part(v, V, vc.data_ptr(), VC, false, true)};
        const bool room = KC.n > 0;                    // (pages of no entry are like no pages)
        check(c.fn, dbs_rotary(parts, 3, dt, Q.b, Q.n, (int32_t)Q.d, (int32_t)table.size(1), table.data_ptr<float>(), table.size(0),
                               pos.data_ptr<int32_t>(), slots.data_ptr<int32_t>(), room ? KC.b : 0, room ? KC.n : 1,
                               truth(a.v[8], false), 0, c.stream));
        if (qg) written(qo);
        written(kc);
        written(vc);
        return wrap(qo);
    });
}

// ---- attention ----

PyObject *tree_attention(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<11> N({"q", "k_cache", "v_cache", "kv_lens", "tree", "tree_lens", "page_table", "scale", "out", "return_lse", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_tree_attention"};
        const Args<11> a(c.fn, N.v, 5, 4, args, nargs, kw);
        const at::Tensor &q = c.need("q", a.v[0]), &k = c.need("k_cache", a.v[1]), &v = c.need("v_cache", a.v[2]);
        const at::Tensor &lens = c.need("kv_lens", a.v[3]);
        const at::Tensor *tree = c.tensor("tree", a.v[4]), *tl = c.tensor("tree_lens", a.v[5]), *pt = c.tensor("page_table", a.v[6]);
        const at::Tensor *given = c.tensor("out", a.v[8]);
        const bool want_lse = truth(a.v[9], false);
        if ((q.scalar_type() != at::kHalf && q.scalar_type() != at::kBFloat16) || q.dim() != 4)
            bad(c.fn, "q has to be float16 or bfloat16 [batch, tokens, q_heads, head_dim]");
        const Heads Q = heads_of(c, "q", q, q.scalar_type());
        if (k.dim() != 4 || k.sizes() != v.sizes()) bad(c.fn, "caches have to be [pages, page_size, kv_heads, head_dim]");
        const Heads K = heads_of(c, "k_cache", k, q.scalar_type()), V = heads_of(c, "v_cache", v, q.scalar_type());
        if (K.d != Q.d || Q.d > 256 || Q.d < 1) bad(c.fn, "the caches' heads have to be like q's, of at most 256 entries");
        if (K.h == 0 || Q.h == 0 || Q.h % K.h || Q.n > 1024) bad(c.fn, "q_heads has to be a multiple of kv_heads, tokens at most 1024");
        dbs_attention_args A{};
        A.dtype = c.type("q", q);
        A.head_dim = (int32_t)Q.d;
        A.q_heads = (int32_t)Q.h;
        A.kv_heads = (int32_t)K.h;
        A.batch = Q.b;
        A.tokens = Q.n;
        A.q = q.data_ptr();
        A.q_batch = Q.sb; A.q_token = Q.sn; A.q_head = Q.sh;
        A.k = k.data_ptr();
        A.v = v.data_ptr();
        A.k_page = K.sb; A.k_entry = K.sn; A.k_head = K.sh;
        A.v_page = V.sb; A.v_entry = V.sn; A.v_head = V.sh;
        A.pages = K.b;
        A.page_size = K.n;
        if (pt) {
            if (pt->dim() != 2) bad(c.fn, "page_table has to be int32 [batch, max_pages]");
            A.max_pages = pt->size(1);
            A.page_row = c.rows("page_table", *pt, Q.b, A.max_pages, at::kInt);
            A.page_table = pt->data_ptr<int32_t>();
        } else {
            if (K.b < Q.b) bad(c.fn, "without a page_table the caches are [batch, entries, kv_heads, head_dim]");
            A.max_pages = 1;
        }
        A.kv_lens = (const int32_t *)c.vector("kv_lens", &lens, Q.b, at::kInt);
        A.tree_lens = (const int32_t *)c.vector("tree_lens", tl, Q.b, at::kInt);
        if (tree) {
            if (tree->scalar_type() != at::kLong || tree->dim() != 3 || tree->size(0) != Q.b || tree->size(1) != Q.n ||
                tree->size(2) != (Q.n + 63) / 64 || !tree->is_contiguous())
                bad(c.fn, "tree has to be contiguous int64 [batch, tokens, ceil(tokens / 64)]");
            A.tree = tree->data_ptr<int64_t>();
        }
        A.scale = (float)real(a.v[7], 1.0 / std::sqrt((double)Q.d));
        c.on(a.v[10]);
        at::Tensor out, lse, scratch;
        if (given) {
            out = *given;
            if (out.sizes() != q.sizes()) bad(c.fn, "out has to have q's shape");
        } else {
            out = c.empty(q.sizes(), q.scalar_type());
        }
        const Heads O = heads_of(c, "out", out, q.scalar_type());
        A.out = out.data_ptr();
        A.o_batch = O.sb; A.o_token = O.sn; A.o_head = O.sh;
        if (want_lse) {
            lse = c.empty({Q.b, Q.n, Q.h}, at::kFloat);
            A.lse = lse.data_ptr<float>();
        }
        check(c.fn, dbs_tree_attention_scratch(&A, &A.scratch_bytes));
        if (A.scratch_bytes > 0) {
            scratch = c.empty({A.scratch_bytes}, at::kByte);
            A.scratch = scratch.data_ptr();
        }
        check(c.fn, dbs_tree_attention(&A, c.stream));
        if (given) written(out);
        if (!want_lse) return wrap(out);
        PyObject *r = PyTuple_New(2);
        if (!r) throw Failed();
        PyTuple_SET_ITEM(r, 0, wrap(out));
        PyTuple_SET_ITEM(r, 1, wrap(lse));
        return r;
    });
}

// ---- logits ----

PyObject *penalize_logits(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<12> N({"logits", "history", "history_lens", "prompt_lens", "repetition", "presence", "frequency", "bias_ids",
                              "bias_vals", "allowed", "out", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_penalize_logits"};
        const Args<12> a(c.fn, N.v, 1, 1, args, nargs, kw);
        const at::Tensor &x = c.need("logits", a.v[0]);
        const at::Tensor *hist = c.tensor("history", a.v[1]), *hl = c.tensor("history_lens", a.v[2]), *pl = c.tensor("prompt_lens", a.v[3]);
        const at::Tensor *rep = c.tensor("repetition", a.v[4]), *pres = c.tensor("presence", a.v[5]), *freq = c.tensor("frequency", a.v[6]);
        const at::Tensor *ids = c.tensor("bias_ids", a.v[7]), *vals = c.tensor("bias_vals", a.v[8]), *allowed = c.tensor("allowed", a.v[9]);
        const at::Tensor *given = c.tensor("out", a.v[10]);
        dbs_logits_args A{};
        A.dtype = c.type("logits", x);
        if (x.dim() != 2) bad(c.fn, "logits have to be [batch, vocab]");
        const int64_t B = x.size(0), V = x.size(1);
        A.batch = B;
        A.vocab = V;
        A.logits = x.data_ptr();
        A.logits_stride = c.rows("logits", x, B, V, x.scalar_type());
        if (hist) {
            if (hist->dim() != 2) bad(c.fn, "history has to be int32 [batch, history_max]");
            A.history_max = hist->size(1);
            A.history_stride = c.rows("history", *hist, B, A.history_max, at::kInt);
            A.history = hist->data_ptr<int32_t>();
        } else if (hl || pl || rep || pres || freq) {
            bad(c.fn, "penalties and lengths need a history");
        }
        if (ids || vals) {
            if (!ids || !vals || ids->dim() != 2) bad(c.fn, "bias_ids int32 and bias_vals float32 [batch, n] come together");
            A.biases = ids->size(1);
            A.bias_stride = c.rows("bias_ids", *ids, B, A.biases, at::kInt);
            if (c.rows("bias_vals", *vals, B, A.biases, at::kFloat) != A.bias_stride && B > 1)
                bad(c.fn, "bias_ids and bias_vals have to have the same strides");
            A.bias_ids = ids->data_ptr<int32_t>();
            A.bias_vals = vals->data_ptr<float>();
        }
        if (allowed) {
            A.allowed_stride = c.rows("allowed", *allowed, B, (V + 31) / 32, at::kInt);
            A.allowed = allowed->data_ptr<int32_t>();
        }
        A.history_lens = (const int32_t *)c.vector("history_lens", hl, B, at::kInt);
        A.prompt_lens = (const int32_t *)c.vector("prompt_lens", pl, B, at::kInt);
        A.repetition = (const float *)c.vector("repetition", rep, B, at::kFloat);
        A.presence = (const float *)c.vector("presence", pres, B, at::kFloat);
        A.frequency = (const float *)c.vector("frequency", freq, B, at::kFloat);
        c.on(a.v[11]);
        const at::Tensor out = given ? *given : c.empty({B, V}, at::kFloat);
        A.out_dtype = c.type("out", out);
        A.out_stride = c.rows("out", out, B, V, out.scalar_type());
        A.out = out.data_ptr();
        check(c.fn, dbs_penalize_logits(&A, c.stream));
        if (given) written(out);
        return wrap(out);
    });
}

// ---- norms with rotation ----

// A head's weight: [head_dim] of any floating type, or none.
dbs_norm_heads normed(Call &c, const char *name, const dbs_rotary_heads &heads, const at::Tensor *w, int64_t d)
{
    dbs_norm_heads H{heads, nullptr, DBS_F32};
    if (w) {
        H.weight_dtype = c.type(name, *w);
        H.weight = c.vector(name, w, d, w->scalar_type());
    }
    return H;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *r = PyTuple_New(2);
    if (!r) throw Failed();
    PyTuple_SET_ITEM(r, 0, a.defined() ? wrap(a) : Py_NewRef(Py_None));
    PyTuple_SET_ITEM(r, 1, b.defined() ? wrap(b) : Py_NewRef(Py_None));
    return r;
}

PyObject *norm_rotary(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<11> N({"q", "k", "q_weight", "k_weight", "table", "positions", "eps", "interleaved", "q_out", "k_out", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_norm_rotary"};
        const Args<11> a(c.fn, N.v, 6, 6, args, nargs, kw);
        const at::Tensor &q = c.need("q", a.v[0]), &table = c.need("table", a.v[4]), &pos = c.need("positions", a.v[5]);
        const at::Tensor *k = c.tensor("k", a.v[1]), *qw = c.tensor("q_weight", a.v[2]), *kw_ = c.tensor("k_weight", a.v[3]);
        const at::Tensor *qg = c.tensor("q_out", a.v[8]), *kg = c.tensor("k_out", a.v[9]);
        const dbs_dtype dt = c.type("q", q);
        const Heads Q = turning(c, q, table, pos, nullptr);
        const Heads K = k ? like(c, "k", *k, q, Q) : Q;
        if (!k && (kw_ || kg)) bad(c.fn, "k_weight and k_out need k");
        c.on(a.v[10]);
        const at::Tensor qo = turned(c, q, qg), ko = k ? turned(c, *k, kg) : at::Tensor();
        dbs_norm_heads parts[2] = {normed(c, "q_weight", part(q, Q, qo.data_ptr(), heads_of(c, "q_out", qo, q.scalar_type()), true, false), qw, Q.d)};
        if (k) parts[1] = normed(c, "k_weight", part(*k, K, ko.data_ptr(), heads_of(c, "k_out", ko, q.scalar_type()), true, false), kw_, Q.d);
        check(c.fn, dbs_norm_rotary(parts, k ? 2 : 1, dt, Q.b, Q.n, (int32_t)Q.d, (int32_t)table.size(1), (float)real(a.v[6], 1e-6),
                                    table.data_ptr<float>(), table.size(0), pos.data_ptr<int32_t>(), nullptr, 0, 1, truth(a.v[7], false), c.stream));
        if (qg) written(qo);
        if (kg) written(ko);
        return pair(qo, ko);
    });
}

PyObject *norm_rotary_append(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<14> N({"q", "k", "v", "q_weight", "k_weight", "table", "positions", "k_cache", "v_cache", "slots", "eps", "interleaved",
                              "q_out", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_norm_rotary_append"};
        const Args<14> a(c.fn, N.v, 10, 10, args, nargs, kw);
        const at::Tensor &q = c.need("q", a.v[0]), &k = c.need("k", a.v[1]), &v = c.need("v", a.v[2]);
        const at::Tensor *qw = c.tensor("q_weight", a.v[3]), *kw_ = c.tensor("k_weight", a.v[4]);
        const at::Tensor &table = c.need("table", a.v[5]), &pos = c.need("positions", a.v[6]);
        const at::Tensor &kc = c.need("k_cache", a.v[7]), &vc = c.need("v_cache", a.v[8]), &slots = c.need("slots", a.v[9]);
        const at::Tensor *qg = c.tensor("q_out", a.v[12]);
        const dbs_dtype dt = c.type("q", q);
        const Heads Q = turning(c, q, table, pos, &slots), K = like(c, "k", k, q, Q), V = like(c, "v", v, q, Q);
        if (kc.dim() != 4 || vc.sizes() != kc.sizes() || K.h != V.h)
            bad(c.fn, "caches have to be [pages, page_size, kv_heads, head_dim]");
        const Heads KC = heads_of(c, "k_cache", kc, q.scalar_type()), VC = heads_of(c, "v_cache", vc, q.scalar_type());
        if (KC.h != K.h || KC.d != Q.d) bad(c.fn, "caches have to have k's heads");
        c.on(a.v[13]);
        const at::Tensor qo = turned(c, q, qg);
        const dbs_norm_heads parts[3] = {
            normed(c, "q_weight", part(q, Q, qo.data_ptr(), heads_of(c, "q_out", qo, q.scalar_type()), true, false), qw, Q.d),
            normed(c, "k_weight", part(k, K, kc.data_ptr(), KC, true, true), kw_, Q.d),
            {part(v, V, vc.data_ptr(), VC, false, true), nullptr, DBS_F32}};
        const bool room = KC.n > 0;                    // (pages of no entry are like no pages)
        check(c.fn, dbs_norm_rotary(parts, 3, dt, Q.b, Q.n, (int32_t)Q.d, (int32_t)table.size(1), (float)real(a.v[10], 1e-6),
                                    table.data_ptr<float>(), table.size(0), pos.data_ptr<int32_t>(), slots.data_ptr<int32_t>(),
                                    room ? KC.b : 0, room ? KC.n : 1, truth(a.v[11], false), c.stream));
        if (qg) written(qo);
        written(kc);
        written(vc);
        return wrap(qo);
    });
}

PyObject *norm_rotary_gradient(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<11> N({"q_grad", "k_grad", "q", "k", "q_weight", "k_weight", "table", "positions", "eps", "interleaved", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_norm_rotary_gradient"};
        const Args<11> a(c.fn, N.v, 8, 8, args, nargs, kw);
        const at::Tensor &qg = c.need("q_grad", a.v[0]), &q = c.need("q", a.v[2]);
        const at::Tensor *kg = c.tensor("k_grad", a.v[1]), *k = c.tensor("k", a.v[3]);
        const at::Tensor *qw = c.tensor("q_weight", a.v[4]), *kw_ = c.tensor("k_weight", a.v[5]);
        const at::Tensor &table = c.need("table", a.v[6]), &pos = c.need("positions", a.v[7]);
        const dbs_dtype dt = c.type("q", q);
        const Heads Q = turning(c, q, table, pos, nullptr);
        if (!k != !kg) bad(c.fn, "k and k_grad come together");
        if (!k && kw_) bad(c.fn, "k_weight needs k");
        c.on(a.v[10]);
        dbs_norm_gradient_heads parts[2] = {};
        at::Tensor dx[2], dw[2];
        for (int p = 0; p < (k ? 2 : 1); ++p) {
            const at::Tensor &x = p ? *k : q, &g = p ? *kg : qg;
            const at::Tensor *w = p ? kw_ : qw;
            const char *name = p ? "k_grad" : "q_grad";
            const Heads X = p ? like(c, "k", x, q, Q) : Q, G = like(c, name, g, q, Q);
            if (G.h != X.h) bad(c.fn, std::string(name) + " has to have its input's heads");
            dx[p] = c.empty(x.sizes(), x.scalar_type());
            dw[p] = c.empty({Q.d}, at::kFloat);
            const Heads O = heads_of(c, "out", dx[p], x.scalar_type());
            const dbs_norm_heads W = normed(c, p ? "k_weight" : "q_weight", dbs_rotary_heads{}, w, Q.d);
            parts[p] = {g.data_ptr(), x.data_ptr(), dx[p].data_ptr(), G.sb, G.sn, G.sh, X.sb, X.sn, X.sh, O.sb, O.sn, O.sh,
                        (int32_t)X.h, W.weight_dtype, W.weight, dw[p].data_ptr<float>()};
        }
        int64_t bytes = 0;
        check(c.fn, dbs_norm_rotary_gradient_scratch(k ? 2 : 1, (int32_t)Q.d, &bytes));
        const at::Tensor scratch = c.empty({bytes}, at::kByte);
        check(c.fn, dbs_norm_rotary_gradient(parts, k ? 2 : 1, dt, Q.b, Q.n, (int32_t)Q.d, (int32_t)table.size(1), (float)real(a.v[8], 1e-6),
                                             table.data_ptr<float>(), table.size(0), pos.data_ptr<int32_t>(), truth(a.v[9], false),
                                             scratch.data_ptr(), bytes, c.stream));
        PyObject *r = PyTuple_New(4);
        if (!r) throw Failed();
        const at::Tensor all[4] = {dx[0], dx[1], dw[0], dw[1]};
        for (int i = 0; i < 4; ++i) PyTuple_SET_ITEM(r, i, all[i].defined() ? wrap(all[i]) : Py_NewRef(Py_None));
        return r;
    });
}

// ---- attention with a window ----

PyObject *window_attention(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<12> N({"q", "k_cache", "v_cache", "kv_lens", "window", "sinks", "q_lens", "page_table", "scale", "out", "return_lse",
                              "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_window_attention"};
        const Args<12> a(c.fn, N.v, 5, 5, args, nargs, kw);
        const at::Tensor &q = c.need("q", a.v[0]), &k = c.need("k_cache", a.v[1]), &v = c.need("v_cache", a.v[2]);
        const at::Tensor &lens = c.need("kv_lens", a.v[3]);
        const at::Tensor *ql = c.tensor("q_lens", a.v[6]), *pt = c.tensor("page_table", a.v[7]), *given = c.tensor("out", a.v[9]);
        const bool want_lse = truth(a.v[10], false);
        if ((q.scalar_type() != at::kHalf && q.scalar_type() != at::kBFloat16) || q.dim() != 4)
            bad(c.fn, "q has to be float16 or bfloat16 [batch, tokens, q_heads, head_dim]");
        const Heads Q = heads_of(c, "q", q, q.scalar_type());
        if (k.dim() != 4 || k.sizes() != v.sizes()) bad(c.fn, "caches have to be [pages, page_size, kv_heads, head_dim]");
        const Heads K = heads_of(c, "k_cache", k, q.scalar_type()), V = heads_of(c, "v_cache", v, q.scalar_type());
        if (K.d != Q.d || Q.d > 256 || Q.d < 1) bad(c.fn, "the caches' heads have to be like q's, of at most 256 entries");
        if (K.h == 0 || Q.h == 0 || Q.h % K.h) bad(c.fn, "q_heads has to be a multiple of kv_heads");
        dbs_window_args A{};
        A.dtype = c.type("q", q);
        A.head_dim = (int32_t)Q.d;
        A.q_heads = (int32_t)Q.h;
        A.kv_heads = (int32_t)K.h;
        A.batch = Q.b;
        A.tokens = Q.n;
        A.q = q.data_ptr();
        A.q_batch = Q.sb; A.q_token = Q.sn; A.q_head = Q.sh;
        A.k = k.data_ptr();
        A.v = v.data_ptr();
        A.k_page = K.sb; A.k_entry = K.sn; A.k_head = K.sh;
        A.v_page = V.sb; A.v_entry = V.sn; A.v_head = V.sh;
        A.pages = K.b;
        A.page_size = K.n;
        if (pt) {
            if (pt->dim() != 2) bad(c.fn, "page_table has to be int32 [batch, max_pages]");
            A.max_pages = pt->size(1);
            A.page_row = c.rows("page_table", *pt, Q.b, A.max_pages, at::kInt);
            A.page_table = pt->data_ptr<int32_t>();
        } else {
            if (K.b < Q.b) bad(c.fn, "without a page_table the caches are [batch, entries, kv_heads, head_dim]");
            A.max_pages = 1;
        }
        A.kv_lens = (const int32_t *)c.vector("kv_lens", &lens, Q.b, at::kInt);
        A.q_lens = (const int32_t *)c.vector("q_lens", ql, Q.b, at::kInt);
        A.window = whole(a.v[4], 0);
        A.sinks = whole(a.v[5], 0);
        if (A.window < 1 || A.sinks < 0) bad(c.fn, "window has to be at least 1, sinks at least 0");
        A.scale = (float)real(a.v[8], 1.0 / std::sqrt((double)Q.d));
        c.on(a.v[11]);
        at::Tensor out, lse, scratch;
        if (given) {
            out = *given;
            if (out.sizes() != q.sizes()) bad(c.fn, "out has to have q's shape");
        } else {
            out = c.empty(q.sizes(), q.scalar_type());
        }
        const Heads O = heads_of(c, "out", out, q.scalar_type());
        A.out = out.data_ptr();
        A.o_batch = O.sb; A.o_token = O.sn; A.o_head = O.sh;
        if (want_lse) {
            lse = c.empty({Q.b, Q.n, Q.h}, at::kFloat);
            A.lse = lse.data_ptr<float>();
        }
        check(c.fn, dbs_window_attention_scratch(&A, &A.scratch_bytes));
        if (A.scratch_bytes > 0) {
            scratch = c.empty({A.scratch_bytes}, at::kByte);
            A.scratch = scratch.data_ptr();
        }
        check(c.fn, dbs_window_attention(&A, c.stream));
        if (given) written(out);
        return want_lse ? pair(out, lse) : wrap(out);
    });
}

// ---- pages of a cache ----

// K and V: [pages, page_size, kv_heads, head_dim] of one layer, or with a dimension of layers before.
dbs_cache_data cache_of(const Call &c, const at::Tensor &k, const at::Tensor &v, int64_t &pages, int64_t &page_size)
{
    const int64_t n = k.dim(), size = (int64_t)k.element_size();
    if ((n != 4 && n != 5) || v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type())
        bad(c.fn, "caches have to be two tensors [pages, page_size, kv_heads, head_dim] or [layers, pages, page_size, kv_heads, head_dim] of one type");
    if (size != 1 && size != 2 && size != 4 && size != 8) bad(c.fn, "entries of caches have to be of 1, 2, 4 or 8 bytes");
    if (k.size(n - 1) > 1 && (k.stride(n - 1) != 1 || v.stride(n - 1) != 1)) bad(c.fn, "caches: the last dimension has to be contiguous");
    pages = k.size(n - 4);
    page_size = k.size(n - 3);
    auto at = [&](const at::Tensor &t, int64_t i) { return t.stride(n - i); };
    const bool layers = n == 5;
    return {k.data_ptr(), v.data_ptr(), layers ? k.size(0) : 1, k.numel() ? k.size(n - 2) : 0, k.size(n - 1), (int32_t)size,   // (without entries: no heads)
            layers ? k.stride(0) : 0, at(k, 4), at(k, 3), at(k, 2), layers ? v.stride(0) : 0, at(v, 4), at(v, 3), at(v, 2)};
}

dbs_page_state state_of(Call &c, const at::Tensor *table, const at::Tensor &lens, const at::Tensor *refs)
{
    dbs_page_state S{};
    if (lens.dim() != 1) bad(c.fn, "kv_lens has to be int32 [batch]");
    S.batch = lens.size(0);
    S.kv_lens = (int32_t *)const_cast<void *>(c.vector("kv_lens", &lens, S.batch, at::kInt));
    if (table) {
        if (table->dim() != 2) bad(c.fn, "page_table has to be int32 [batch, max_pages]");
        S.max_pages = table->size(1);
        S.page_row = c.rows("page_table", *table, S.batch, S.max_pages, at::kInt);
        S.page_table = table->data_ptr<int32_t>();
    }
    if (refs) {
        if (refs->dim() != 1) bad(c.fn, "refs has to be int32 [pages]");
        S.pages = refs->size(0);
        S.refs = (int32_t *)const_cast<void *>(c.vector("refs", refs, S.pages, at::kInt));
    }
    return S;
}

PyObject *cache_resize(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<7> N({"page_table", "kv_lens", "refs", "lens", "page_size", "columns", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_cache_resize"};
        const Args<7> a(c.fn, N.v, 5, 5, args, nargs, kw);
        const at::Tensor &table = c.need("page_table", a.v[0]), &kv = c.need("kv_lens", a.v[1]), &refs = c.need("refs", a.v[2]);
        const at::Tensor &lens = c.need("lens", a.v[3]);
        dbs_page_state S = state_of(c, &table, kv, &refs);
        S.page_size = whole(a.v[4], 0);
        const int64_t columns = whole(a.v[5], 0);
        if (S.page_size < 1 || columns < 0) bad(c.fn, "page_size has to be at least 1, columns at least 0");
        const int32_t *want = (const int32_t *)c.vector("lens", &lens, S.batch, at::kInt);
        c.on(a.v[6]);
        int64_t bytes = 0;
        check(c.fn, dbs_cache_resize_scratch(&S, columns, &bytes));
        const at::Tensor status = c.empty({S.batch}, at::kInt);
        at::Tensor slots, scratch;
        if (a.v[5]) slots = c.empty({S.batch, columns}, at::kInt);
        if (bytes > 0) scratch = c.empty({bytes}, at::kByte);
        check(c.fn, dbs_cache_resize(&S, want, status.data_ptr<int32_t>(), slots.defined() ? slots.data_ptr<int32_t>() : nullptr, columns,
                                     scratch.defined() ? scratch.data_ptr() : nullptr, bytes, c.stream));
        written(table);
        written(kv);
        written(refs);
        return pair(status, slots);
    });
}

PyObject *cache_fork(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<8> N({"k_cache", "v_cache", "page_table", "kv_lens", "refs", "parents", "children", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_cache_fork"};
        const Args<8> a(c.fn, N.v, 7, 7, args, nargs, kw);
        const at::Tensor &k = c.need("k_cache", a.v[0]), &v = c.need("v_cache", a.v[1]);
        const at::Tensor &table = c.need("page_table", a.v[2]), &kv = c.need("kv_lens", a.v[3]), &refs = c.need("refs", a.v[4]);
        const at::Tensor &from = c.need("parents", a.v[5]), &to = c.need("children", a.v[6]);
        int64_t pages = 0, page_size = 0;
        const dbs_cache_data D = cache_of(c, k, v, pages, page_size);
        dbs_page_state S = state_of(c, &table, kv, &refs);
        if (S.pages != pages) bad(c.fn, "refs has to have a count for each page of the caches");
        if (page_size < 1) bad(c.fn, "pages have to hold an entry at least");
        S.page_size = page_size;
        if (from.dim() != 1) bad(c.fn, "parents and children have to be int32 [n]");
        const int64_t n = from.size(0);
        const int32_t *p = (const int32_t *)c.vector("parents", &from, n, at::kInt), *ch = (const int32_t *)c.vector("children", &to, n, at::kInt);
        c.on(a.v[7]);
        int64_t bytes = 0;
        check(c.fn, dbs_cache_fork_scratch(&S, n, &bytes));
        const at::Tensor status = c.empty({n}, at::kInt), scratch = c.empty({bytes}, at::kByte);
        check(c.fn, dbs_cache_fork(&D, &S, p, ch, n, status.data_ptr<int32_t>(), scratch.data_ptr(), bytes, c.stream));
        for (const at::Tensor *t : {&k, &v, &table, &kv, &refs}) written(*t);
        return wrap(status);
    });
}

PyObject *cache_compact(PyObject *, PyObject *const *args, Py_ssize_t nargs, PyObject *kw)
{
    static const Names<8> N({"k_cache", "v_cache", "kv_lens", "tree_lens", "accepted", "accepted_lens", "page_table", "stream"});
    return guarded([&]() -> PyObject * {
        Call c{"dbs_cache_compact"};
        const Args<8> a(c.fn, N.v, 6, 5, args, nargs, kw);
        const at::Tensor &k = c.need("k_cache", a.v[0]), &v = c.need("v_cache", a.v[1]), &kv = c.need("kv_lens", a.v[2]);
        const at::Tensor &tree = c.need("tree_lens", a.v[3]), &acc = c.need("accepted", a.v[4]);
        const at::Tensor *al = c.tensor("accepted_lens", a.v[5]), *table = c.tensor("page_table", a.v[6]);
        int64_t pages = 0, page_size = 0;
        const dbs_cache_data D = cache_of(c, k, v, pages, page_size);
        dbs_page_state S = state_of(c, table, kv, nullptr);
        S.pages = pages;
        if (!table) {
            if (pages < S.batch) bad(c.fn, "without a page_table the caches are [batch, entries, kv_heads, head_dim]");
            S.max_pages = 1;
        }
        if (page_size == 0 || pages == 0) S.max_pages = 0;              // (no room, whatever the table says)
        S.page_size = page_size > 0 ? page_size : 1;
        if (acc.dim() != 2) bad(c.fn, "accepted has to be int32 [batch, n]");
        const int64_t stride = c.rows("accepted", acc, S.batch, acc.size(1), at::kInt);
        const int32_t *tl = (const int32_t *)c.vector("tree_lens", &tree, S.batch, at::kInt);
        const int32_t *n = (const int32_t *)c.vector("accepted_lens", al, S.batch, at::kInt);
        c.on(a.v[7]);
        const at::Tensor lens = c.empty({S.batch}, at::kInt);
        check(c.fn, dbs_cache_compact(&D, &S, tl, acc.data_ptr<int32_t>(), acc.size(1), stride, n, lens.data_ptr<int32_t>(), c.stream));
        written(k);
        written(v);
        return wrap(lens);
    });
}

PyObject *set_error(PyObject *, PyObject *e)
{
    Py_XDECREF(g_error);
    g_error = Py_NewRef(e);
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL | METH_KEYWORDS

PyMethodDef g_methods[] = {
    {"w4_linear", FAST(w4_linear),
     "w4_linear(x, q, scales, zeros=None, *, group=128, y=None, stream=None)\n--\n\n"
     "dbs_w4_linear: y[t, i] = sum_j x[t, j] (q[i, j] - z[i, j // group]) s[i, j // group].\n\n"
     "x [tokens, n] or [n], float32, float16 or bfloat16; q uint8 [m, ceil(n/2)]\n"
     "(column 2c in the low half of byte c); scales [m, ceil(n/group)] in any of\n"
     "those types; zeros uint8 of the same shape, or None for 8.  Rows of q that\n"
     "start on 16-byte boundaries are the fast case.  Returns y [tokens, m] (or\n"
     "[m]) in x's type."},
    {"rotary_table", FAST(rotary_table),
     "rotary_table(positions, dim, *, base=10000.0, scaling=None, factor=1.0, trained=0.0, beta_fast=32.0, beta_slow=1.0, "
     "device=None, stream=None)\n--\n\n"
     "dbs_rotary_table: float32 [positions, dim], cosines then sines.\n"
     "scaling: None, \"linear\", \"ntk\" or \"yarn\" (with `trained` positions)."},
    {"rotary", FAST(rotary),
     "rotary(q, k, table, positions, *, interleaved=False, transposed=False, q_out=None, k_out=None, stream=None)\n--\n\n"
     "dbs_rotary: q and k (or None) [batch, tokens, heads, head_dim] or [tokens,\n"
     "heads, head_dim], turned by their tokens' positions (int32).  The first\n"
     "table.shape[1] entries of a head are turned, in pairs (i, i + dim/2) or,\n"
     "interleaved, (2i, 2i + 1); the rest is copied.  transposed turns the other\n"
     "way: the gradient.  Returns (q, k), new tensors unless q_out and k_out are\n"
     "given (the inputs themselves: in place)."},
    {"rotary_append", FAST(rotary_append),
     "rotary_append(q, k, v, table, positions, k_cache, v_cache, slots, *, interleaved=False, q_out=None, stream=None)\n--\n\n"
     "dbs_rotary with a cache: q is turned and returned; k, turned, and v go to\n"
     "entry slots[token] (int32; outside the cache: not written) of k_cache and\n"
     "v_cache [pages, page_size, kv_heads, head_dim], in the same launch."},
    {"tree_attention", FAST(tree_attention),
     "tree_attention(q, k_cache, v_cache, kv_lens, tree=None, *, tree_lens=None, page_table=None, scale=None, out=None, "
     "return_lse=False, stream=None)\n--\n\n"
     "dbs_tree_attention: drafted tokens q [batch, tokens, q_heads, head_dim]\n"
     "(float16 or bfloat16) against caches [pages, page_size, kv_heads, head_dim]\n"
     "with page_table int32 [batch, max_pages], or, without one, [batch, entries,\n"
     "kv_heads, head_dim].  kv_lens int32 [batch] counts a sequence's entries, its\n"
     "drafted tokens last among them; tree_lens int32 [batch] counts those (None:\n"
     "all of q's tokens).  tree int64 [batch, tokens, ceil(tokens / 64)]: bit i of\n"
     "token t's words is set if it sees drafted token i (None: i <= t).  Returns\n"
     "out like q, and with return_lse the float32 [batch, tokens, q_heads]\n"
     "logarithm of each row's sum."},
    {"penalize_logits", FAST(penalize_logits),
     "penalize_logits(logits, *, history=None, history_lens=None, prompt_lens=None, repetition=None, presence=None, "
     "frequency=None, bias_ids=None, bias_vals=None, allowed=None, out=None, stream=None)\n--\n\n"
     "dbs_penalize_logits: logits [batch, vocab] (float32, float16, bfloat16) with\n"
     "the penalties of the tokens in history int32 [batch, history_max]\n"
     "(history_lens int32 [batch] of them; the first prompt_lens[b] count for\n"
     "repetition alone), biases float32 bias_vals at int32 bias_ids [batch, n], and\n"
     "-inf where bit v % 32 of allowed int32 [batch, ceil(vocab / 32)] is clear.\n"
     "repetition, presence and frequency: float32 [batch].  Returns float32, or\n"
     "`out` (which may be logits: in place)."},
    {"norm_rotary", FAST(norm_rotary),
     "norm_rotary(q, k, q_weight, k_weight, table, positions, *, eps=1e-6, interleaved=False, q_out=None, k_out=None, stream=None)\n--\n\n"
     "dbs_norm_rotary: rotary of heads that are divided by the root of their mean\n"
     "square (plus eps) and multiplied by a weight [head_dim] (float32, float16 or\n"
     "bfloat16; None: ones), each head of q and k (or None) by its own.  Returns\n"
     "(q, k) as rotary does."},
    {"norm_rotary_append", FAST(norm_rotary_append),
     "norm_rotary_append(q, k, v, q_weight, k_weight, table, positions, k_cache, v_cache, slots, *, eps=1e-6, interleaved=False, "
     "q_out=None, stream=None)\n--\n\n"
     "dbs_norm_rotary with a cache: rotary_append of normed q and k; v is copied."},
    {"norm_rotary_gradient", FAST(norm_rotary_gradient),
     "norm_rotary_gradient(q_grad, k_grad, q, k, q_weight, k_weight, table, positions, *, eps=1e-6, interleaved=False, stream=None)\n--\n\n"
     "dbs_norm_rotary_gradient: from the gradients of norm_rotary's results and its\n"
     "inputs (k_grad and k may be None) the gradients of q, k (in their type),\n"
     "q_weight and k_weight (float32 [head_dim])."},
    {"window_attention", FAST(window_attention),
     "window_attention(q, k_cache, v_cache, kv_lens, window, *, sinks=0, q_lens=None, page_table=None, scale=None, out=None, "
     "return_lse=False, stream=None)\n--\n\n"
     "dbs_window_attention: q [batch, tokens, q_heads, head_dim] (float16 or\n"
     "bfloat16), one token or a whole prompt, against caches as tree_attention takes\n"
     "them.  The last q_lens[b] (None: all of q's tokens) of a sequence's kv_lens[b]\n"
     "entries are its tokens; one at position p sees the entries j <= p with\n"
     "p - j < window or j < sinks.  Returns out like q, and with return_lse the\n"
     "float32 [batch, tokens, q_heads] logarithm of each row's sum."},
    {"cache_resize", FAST(cache_resize),
     "cache_resize(page_table, kv_lens, refs, lens, page_size, *, columns=None, stream=None)\n--\n\n"
     "dbs_cache_resize: sequence b gets length lens[b] (below 0: as it is) by giving\n"
     "back pages or taking free ones, lowest numbers first.  page_table int32 [batch,\n"
     "max_pages], kv_lens int32 [batch] and refs int32 [pages] (how many sequences own\n"
     "a page) are changed in place.  Returns (status, slots): status int32 [batch], 0\n"
     "or why a sequence kept its length (1 no free page, 2 its last page is shared, 3\n"
     "too long for its row); slots int32 [batch, columns], where the first `columns`\n"
     "new entries go (-1: nowhere), or None."},
    {"cache_fork", FAST(cache_fork),
     "cache_fork(k_cache, v_cache, page_table, kv_lens, refs, parents, children, *, stream=None)\n--\n\n"
     "dbs_cache_fork: the empty sequences children (int32 [n]) become copies of\n"
     "parents: full pages are shared, the entries of a last page that is not full are\n"
     "copied to a free one.  Caches [pages, page_size, kv_heads, head_dim], or with a\n"
     "first dimension of layers.  Returns status int32 [n]: 0, 1 no free page, 2 not\n"
     "an empty sequence, or listed before."},
    {"cache_compact", FAST(cache_compact),
     "cache_compact(k_cache, v_cache, kv_lens, tree_lens, accepted, accepted_lens=None, *, page_table=None, stream=None)\n--\n\n"
     "dbs_cache_compact: of a sequence's last tree_lens[b] entries, its drafted\n"
     "tokens, those numbered accepted[b] (int32 [batch, n], ascending; accepted_lens[b]\n"
     "of them, the first that does not ascend ends the list) move to the front.  Caches\n"
     "as of cache_fork, or without a page_table [batch, entries, kv_heads, head_dim].\n"
     "Returns the new lengths; kv_lens and the pages stay (cache_resize takes both on)."},
    {"_set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_dbsops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dbsops(void) { return PyModule_Create(&g_module); }
