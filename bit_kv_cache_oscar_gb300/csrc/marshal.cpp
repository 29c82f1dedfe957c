// The Python side of the INT4 entry points: every argument's type, shape and device checked, addresses,
// strides and the current stream passed on to liboscar.so: the one that the binding loaded, whose entry points
// connect() looks up, since a library found by name or path could be another copy of the package.
//
// These calls are made once per layer and token.  Checked in Python one costs 12 to 20 us of host time, more
// than most of the kernels it starts take at batch 1; here it costs about 1 us.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <dlfcn.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <exception>
#include <initializer_list>
#include <string>

#include "oscar_int4.h"

namespace {

PyObject *g_error = nullptr;                 // OscarError

// liboscar.so's entry points (connect)
#define ENTRY_POINTS(X) \
    X(oscar_append_kv) X(oscar_demote_int4) X(oscar_promote_int4) X(oscar_decode_attention_int4) X(oscar_attention_mass_int4) X(oscar_evict_int4) \
    X(oscar_last_error_string)
struct {
#define X(f) decltype(&::f) f;
    ENTRY_POINTS(X)
#undef X
} g_lib;
PyObject *s_k, *s_v, *s_codes_k, *s_codes_v, *s_scale_zero, *s_m, *s_l, *s_acc, *s_n_splits, *s_device, *s_index, *s_cuda_stream;
PyObject *s_head_dim, *s_n_kv_heads, *s_gqa, *s_page_size, *s_group, *s_sink, *s_recent, *s_levels_k, *s_levels_v;

struct Refused : std::exception {};          // a Python error is set

[[noreturn]] void refuse(const std::string &text) {
    PyErr_SetString(g_error, text.c_str());
    throw Refused();
}

std::string shape_text(c10::ArrayRef<int64_t> s) {
    std::string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
const char *dtype_text(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kByte: return "torch.uint8";
        default: return c10::toString(t);
    }
}

using Shape = std::initializer_list<int64_t>;

struct Attr {                                // an attribute, held while its address is used
    PyObject *o;
    Attr(PyObject *from, PyObject *name) : o(PyObject_GetAttr(from, name)) {
        if (!o) throw Refused();
    }
    ~Attr() { Py_DECREF(o); }
    Attr(const Attr &) = delete;
};
double real(PyObject *o) {
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Refused();
    return x;
}
int32_t whole(PyObject *o) {
    const long x = PyLong_AsLong(o);
    if (x == -1 && PyErr_Occurred()) throw Refused();
    if (x != (int32_t)x) refuse("an integer argument passes 32 bits");
    return (int32_t)x;
}

// The fields of a Layout, read on every call: an object that is copied, sent to another process or used by
// several threads holds nothing of this extension.
oscar_layout_t layout(PyObject *o) {
    oscar_layout_t L = {};
    const auto field = [&](PyObject *name) { return whole(Attr(o, name).o); };
    L.head_dim = field(s_head_dim);
    L.n_kv_heads = field(s_n_kv_heads);
    L.gqa = field(s_gqa);
    L.page_size = field(s_page_size);
    L.group = field(s_group);
    L.sink = field(s_sink);
    L.recent = field(s_recent);
    const Attr k(o, s_levels_k), v(o, s_levels_v);
    if (k.o == Py_None && v.o == Py_None) return L;
    const auto levels = [](PyObject *from, float *to) {
        if (!PySequence_Check(from) || PySequence_Size(from) != 4) refuse("a layout's levels are 4 numbers for keys and 4 for values, or None");
        for (int i = 0; i < 4; ++i) {
            PyObject *x = PySequence_GetItem(from, i);
            if (!x) throw Refused();
            const double d = PyFloat_AsDouble(x);
            Py_DECREF(x);
            if (d == -1.0 && PyErr_Occurred()) throw Refused();
            to[i] = (float)d;
        }
    };
    levels(k.o, L.levels_k);
    levels(v.o, L.levels_v);
    return L;
}

struct Call {
    std::string name;
    int dev = 0;
    explicit Call(const char *n) : name(n) {
        try {
            dev = c10::cuda::current_device();
        } catch (const std::exception &) {
            refuse("no current CUDA device");
        }
    }
    const at::Tensor &tensor(const char *what, PyObject *o) const {
        if (!THPVariable_Check(o)) refuse(name + ": " + what + " must be a tensor");
        return THPVariable_Unpack(o);
    }
    void check(const char *what, const at::Tensor &t, at::ScalarType type, Shape shape) const {
        const c10::ArrayRef<int64_t> want(shape.begin(), shape.size());
        if (t.scalar_type() != type) refuse(name + ": " + what + " must be " + dtype_text(type) + ", not " + dtype_text(t.scalar_type()));
        if (t.sizes() != want) refuse(name + ": " + what + " must have shape " + shape_text(want) + ", not " + shape_text(t.sizes()));
        if (!t.is_cuda() || t.device().index() != dev) refuse(name + ": " + what + " is on " + t.device().str() + ", not on the current CUDA device");
    }
    // address of a contiguous tensor (None: NULL)
    template <typename T>
    T *at(const char *what, PyObject *o, at::ScalarType type, Shape shape) const {
        if (o == Py_None) return nullptr;
        const at::Tensor &t = tensor(what, o);
        check(what, t, type, shape);
        if (!t.is_contiguous()) refuse(name + ": " + what + " must be contiguous");
        return static_cast<T *>(t.data_ptr());
    }
    const int32_t *ints(const char *what, PyObject *o, int64_t n) const { return at<int32_t>(what, o, at::kInt, {n}); }
    // [n, heads, 128] whose heads of one token lie together: address and token stride
    const uint16_t *heads(const char *what, PyObject *o, int64_t n, int64_t heads, int64_t *stride) const {
        const at::Tensor &t = tensor(what, o);
        check(what, t, at::kBFloat16, {n, heads, 128});
        if (n && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != 128)))
            refuse(name + ": the heads of one token of " + what + " must lie together");
        *stride = n > 1 ? t.stride(0) : heads * 128;
        return static_cast<const uint16_t *>(t.data_ptr());
    }
    oscar_bf16_pool_t bf16(const oscar_layout_t *L, PyObject *pool) const {
        const Attr k(pool, s_k), v(pool, s_v);
        const at::Tensor &t = tensor("pool k", k.o);
        const int64_t n = t.dim() ? t.size(0) : 0;
        return {at<uint16_t>("pool k", k.o, at::kBFloat16, {n, L->page_size, L->n_kv_heads, 128}),
                at<uint16_t>("pool v", v.o, at::kBFloat16, {n, L->page_size, L->n_kv_heads, 128}), pages32(n)};
    }
    oscar_int4_pool_t int4(const oscar_layout_t *L, PyObject *pool) const {
        const Attr k(pool, s_codes_k), v(pool, s_codes_v), z(pool, s_scale_zero);
        const at::Tensor &t = tensor("codes_k", k.o);
        const int64_t n = t.dim() ? t.size(0) : 0, H = L->n_kv_heads, ps = L->page_size;
        if (L->group < 1) refuse(name + ": group " + std::to_string(L->group));
        return {at<uint8_t>("codes_k", k.o, at::kByte, {n, H, ps, 64}), at<uint8_t>("codes_v", v.o, at::kByte, {n, H, ps, 64}),
                at<uint16_t>("scale_zero", z.o, at::kBFloat16, {n, H, ps, 128 / L->group, 4}), pages32(n)};
    }
    // [batch, max_pages] of a page table
    void table(PyObject *o, int64_t *batch, int64_t *max_pages) const {
        const at::Tensor &t = tensor("page table", o);
        if (t.dim() != 2) refuse(name + ": page tables must be [batch, max_pages]");
        *batch = t.size(0);
        *max_pages = t.size(1);
    }
    const int32_t *pages(const char *what, PyObject *o, int64_t batch, int64_t max_pages) const {
        return at<int32_t>(what, o, at::kInt, {batch, max_pages});
    }
    void *stream(PyObject *o) const {
        if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
        const Attr d(o, s_device), i(d.o, s_index), s(o, s_cuda_stream);
        if (PyLong_AsLong(i.o) != dev) refuse(name + ": the stream is not one of the current CUDA device");
        void *p = PyLong_AsVoidPtr(s.o);
        if (PyErr_Occurred()) throw Refused();
        return p;
    }
    int32_t pages32(int64_t n) const {
        if (n > 2147483647) refuse(name + ": more than 2^31 - 1 pages or requests");
        return (int32_t)n;
    }
    void done(oscar_status_t st) const {
        if (st != OSCAR_OK) refuse(name + " failed (" + std::to_string((int)st) + "): " + g_lib.oscar_last_error_string());
    }
};

// The interpreter's lock is given up for a call into the library; every argument is formed before.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};
template <typename F, typename... A>
oscar_status_t unlocked(F f, A... args) {
    const Unlocked u;
    return f(args...);
}

// layout, q, k, v, pool, page_table, req_idx, positions, q_out, q_weight, k_weight, eps, rope, rot_dim, interleaved,
// rope_positions, stream
void append_kv(PyObject *const *a) {
    const oscar_layout_t layout_ = layout(a[0]), *L = &layout_;
    const Call c("oscar_append_kv");
    const int64_t H = L->n_kv_heads, Hq = H * L->gqa;
    const at::Tensor &k = c.tensor("k", a[2]);
    const int64_t n = k.dim() ? k.size(0) : 0;
    int64_t qs = 0, ks, vs, batch, max_pages;
    const uint16_t *qp = a[1] == Py_None ? nullptr : c.heads("q", a[1], n, Hq, &qs);
    const uint16_t *kp = c.heads("k", a[2], n, H, &ks), *vp = c.heads("v", a[3], n, H, &vs);
    const oscar_bf16_pool_t pool = c.bf16(L, a[4]);
    c.table(a[5], &batch, &max_pages);
    const int32_t *pt = c.pages("page_table", a[5], batch, max_pages), *req = c.ints("req_idx", a[6], n), *pos = c.ints("positions", a[7], n);
    uint16_t *qo = c.at<uint16_t>("q_out", a[8], at::kBFloat16, {n, Hq, 128});
    const uint16_t *wq = c.at<uint16_t>("q_weight", a[9], at::kBFloat16, {128}), *wk = c.at<uint16_t>("k_weight", a[10], at::kBFloat16, {128});
    int64_t rows = 0;
    if (a[12] != Py_None) {
        const at::Tensor &r = c.tensor("rope", a[12]);
        rows = r.dim() ? r.size(0) : 0;
    }
    const float *rope = c.at<float>("rope", a[12], at::kFloat, {rows, 128});
    const int turn = PyObject_IsTrue(a[14]);
    if (turn < 0) throw Refused();
    const int32_t *rp = c.ints("rope_positions", a[15], n), rot = whole(a[13]);
    const float eps = (float)real(a[11]);
    void *st = c.stream(a[16]);
    c.done(unlocked(g_lib.oscar_append_kv, L, qp, qs, kp, ks, vp, vs, c.pages32(n), wq, wk, eps, rope, (int32_t)std::min<int64_t>(rows, 2147483647),
                                   rot, turn, &pool, pt, c.pages32(max_pages), c.pages32(batch), req, pos, rp, qo, st));
}

// layout, src, bf16_page_table, dst, int4_page_table, pos_begin, pos_end, c_K, c_V, stream
void demote_int4(PyObject *const *a) {
    const oscar_layout_t layout_ = layout(a[0]), *L = &layout_;
    const Call c("oscar_demote_int4");
    int64_t batch, max_pages;
    c.table(a[4], &batch, &max_pages);
    const oscar_bf16_pool_t src = c.bf16(L, a[1]);
    const oscar_int4_pool_t dst = c.int4(L, a[3]);
    const int32_t *bpt = c.pages("bf16_page_table", a[2], batch, max_pages), *ipt = c.pages("int4_page_table", a[4], batch, max_pages);
    const int32_t *lo = c.ints("pos_begin", a[5], batch), *hi = c.ints("pos_end", a[6], batch);
    const float ck = (float)real(a[7]), cv = (float)real(a[8]);
    void *st = c.stream(a[9]);
    c.done(unlocked(g_lib.oscar_demote_int4, L, &src, bpt, &dst, ipt, c.pages32(max_pages), c.pages32(batch), lo, hi, ck, cv, st));
}

// layout, src, int4_page_table, dst, bf16_page_table, pos_begin, pos_end, stream
void promote_int4(PyObject *const *a) {
    const oscar_layout_t layout_ = layout(a[0]), *L = &layout_;
    const Call c("oscar_promote_int4");
    int64_t batch, max_pages;
    c.table(a[2], &batch, &max_pages);
    const oscar_int4_pool_t src = c.int4(L, a[1]);
    const oscar_bf16_pool_t dst = c.bf16(L, a[3]);
    const int32_t *ipt = c.pages("int4_page_table", a[2], batch, max_pages), *bpt = c.pages("bf16_page_table", a[4], batch, max_pages);
    const int32_t *lo = c.ints("pos_begin", a[5], batch), *hi = c.ints("pos_end", a[6], batch);
    void *st = c.stream(a[7]);
    c.done(unlocked(g_lib.oscar_promote_int4, L, &src, ipt, &dst, bpt, c.pages32(max_pages), c.pages32(batch), lo, hi, st));
}

// what decode attention and the attention weights share: layout, q, bf16_pool, bf16_page_table, int4_pool,
// int4_page_table, seq_len, hist_end, sm_scale
struct Attention {
    oscar_layout_t layout_;
    const oscar_layout_t *L = &layout_;
    int64_t batch, max_pages, Hq;
    const uint16_t *q;
    oscar_bf16_pool_t bf;
    oscar_int4_pool_t i4;
    const int32_t *bpt, *ipt, *T, *he;
    float scale;
    const Call call;
    Attention(const Attention &) = delete;
    Attention(const char *name, PyObject *const *a) : layout_(layout(a[0])), call(name) {
        const Call &c = call;
        c.table(a[5], &batch, &max_pages);
        Hq = (int64_t)L->n_kv_heads * L->gqa;
        q = c.at<uint16_t>("q", a[1], at::kBFloat16, {batch, Hq, 128});
        bf = c.bf16(L, a[2]);
        bpt = c.pages("bf16_page_table", a[3], batch, max_pages);
        i4 = c.int4(L, a[4]);
        ipt = c.pages("int4_page_table", a[5], batch, max_pages);
        T = c.ints("seq_len", a[6], batch);
        he = c.ints("hist_end", a[7], batch);
        scale = (float)real(a[8]);
    }
};

// ..., partials, out, out_f32, lse, merge_counters, stream
void decode_attention_int4(PyObject *const *a) {
    const Attention x("oscar_decode_attention_int4", a);
    const Call &c = x.call;
    const Attr m(a[9], s_m), l(a[9], s_l), acc(a[9], s_acc), ns(a[9], s_n_splits);
    const int32_t S = whole(ns.o);
    const int64_t S1 = (int64_t)S + 1;
    const oscar_partials_t part{c.at<float>("partials m", m.o, at::kFloat, {x.batch, x.Hq, S1}), c.at<float>("partials l", l.o, at::kFloat, {x.batch, x.Hq, S1}),
                                c.at<float>("partials acc", acc.o, at::kFloat, {x.batch, x.Hq, S1, 128}), S};
    uint16_t *out = c.at<uint16_t>("out", a[10], at::kBFloat16, {x.batch, x.Hq, 128});
    float *of = c.at<float>("out_f32", a[11], at::kFloat, {x.batch, x.Hq, 128}), *lse = c.at<float>("lse", a[12], at::kFloat, {x.batch, x.Hq});
    int32_t *counters = c.at<int32_t>("merge_counters", a[13], at::kInt, {x.batch * x.L->n_kv_heads});
    void *st = c.stream(a[14]);
    c.done(unlocked(g_lib.oscar_decode_attention_int4, x.L, x.q, &x.bf, x.bpt, &x.i4, x.ipt, c.pages32(x.max_pages), x.T, x.he, c.pages32(x.batch), x.scale,
                                               &part, out, of, lse, counters, st));
}

// ..., lse, mass, stream
void attention_mass_int4(PyObject *const *a) {
    const Attention x("oscar_attention_mass_int4", a);
    const Call &c = x.call;
    const float *lse = c.at<float>("lse", a[9], at::kFloat, {x.batch, x.Hq});
    float *mass = c.at<float>("mass", a[10], at::kFloat, {x.batch, x.L->n_kv_heads, x.max_pages * x.L->page_size});
    void *st = c.stream(a[11]);
    c.done(unlocked(g_lib.oscar_attention_mass_int4, x.L, x.q, &x.bf, x.bpt, &x.i4, x.ipt, c.pages32(x.max_pages), x.T, x.he, c.pages32(x.batch), x.scale, lse,
                                             mass, st));
}

// layout, src, src_page_table, dst, dst_page_table, seq_len, hist_end, keep, mass, mass_out, kept, stream
void evict_int4(PyObject *const *a) {
    const oscar_layout_t layout_ = layout(a[0]), *L = &layout_;
    const Call c("oscar_evict_int4");
    int64_t batch, max_pages;
    c.table(a[2], &batch, &max_pages);
    const oscar_int4_pool_t src = c.int4(L, a[1]), dst = c.int4(L, a[3]);
    const int32_t *spt = c.pages("src_page_table", a[2], batch, max_pages), *dpt = c.pages("dst_page_table", a[4], batch, max_pages);
    const int32_t *T = c.ints("seq_len", a[5], batch), *he = c.ints("hist_end", a[6], batch), *keep = c.ints("keep", a[7], batch);
    const int64_t H = L->n_kv_heads, N = max_pages * L->page_size;
    const float *mass = c.at<float>("mass", a[8], at::kFloat, {batch, H, N});
    float *out = c.at<float>("mass_out", a[9], at::kFloat, {batch, H, N});
    const at::Tensor &k = c.tensor("kept", a[10]);
    const int64_t stride = k.dim() ? k.size(k.dim() - 1) : 0;
    int32_t *kept = c.at<int32_t>("kept", a[10], at::kInt, {batch, H, stride});
    void *st = c.stream(a[11]);
    c.done(unlocked(g_lib.oscar_evict_int4, L, &src, spt, &dst, dpt, c.pages32(max_pages), c.pages32(batch), T, he, keep, mass, out, kept, c.pages32(stride), st));
}

// Python entry: a fixed number of positional arguments; no C++ exception leaves it.
template <void (*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != N) return PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", N, n);
    try {
        F(args);
    } catch (const Refused &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(g_error, e.what());
        return nullptr;
    }
    Py_RETURN_NONE;
}

// connect(handle of the loaded liboscar.so, the exception class that refusals raise): before any other call
PyObject *connect(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 2) return PyErr_Format(PyExc_TypeError, "2 arguments, not %zd", n);
    void *lib = PyLong_AsVoidPtr(args[0]);
    if (PyErr_Occurred()) return nullptr;
#define X(f)                                                                                     \
    g_lib.f = lib ? reinterpret_cast<decltype(&::f)>(dlsym(lib, #f)) : nullptr;                  \
    if (!g_lib.f) return PyErr_Format(PyExc_ImportError, "liboscar.so has no " #f);
    ENTRY_POINTS(X)
#undef X
    Py_XSETREF(g_error, Py_NewRef(args[1]));
    Py_RETURN_NONE;
}

#define ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(append_kv, 17), ENTRY(demote_int4, 10), ENTRY(promote_int4, 8), ENTRY(decode_attention_int4, 15),
                           ENTRY(attention_mass_int4, 12), ENTRY(evict_int4, 12), 
                           {"connect", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&connect)), METH_FASTCALL, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", "Argument checks of the INT4 entry points.", -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) {
    struct { PyObject **to; const char *text; } names[] = {
        {&s_k, "k"}, {&s_v, "v"}, {&s_codes_k, "codes_k"}, {&s_codes_v, "codes_v"}, {&s_scale_zero, "scale_zero"}, {&s_m, "m"}, {&s_l, "l"},
        {&s_acc, "acc"}, {&s_n_splits, "n_splits"}, {&s_device, "device"}, {&s_index, "index"}, {&s_cuda_stream, "cuda_stream"},
        {&s_head_dim, "head_dim"}, {&s_n_kv_heads, "n_kv_heads"}, {&s_gqa, "gqa"}, {&s_page_size, "page_size"}, {&s_group, "group"},
        {&s_sink, "sink"}, {&s_recent, "recent"}, {&s_levels_k, "levels_k"}, {&s_levels_v, "levels_v"}};
    for (auto &n : names)
        if (!(*n.to = PyUnicode_InternFromString(n.text))) return nullptr;
    PyObject *m = PyModule_Create(&g_module);
    if (!m) return nullptr;
    g_error = Py_NewRef(PyExc_RuntimeError);
    return m;
}
