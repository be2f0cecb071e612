// binding.cpp -- the cache-side calls and spec_rollback as Python functions: checks of the torch tensors, then one call
// into libspecverify.so.  The same checks written in Python cost 12 to 15 us a call on the host that
// drives a GB300, more than several of the kernels run.
//
// Every function returns the library's status; a wrong tensor raises ValueError.  The library's entry
// points arrive as addresses through init(), so that this module and the ctypes binding drive one
// loaded library.
#include <torch/csrc/autograd/python_variable.h>

#include <c10/core/ScalarType.h>

#include <cstdarg>

#include "../../include/spec_cache.h"

namespace {

struct Entry {
    decltype(&spec_append) append;
    decltype(&spec_attention) attention;
    decltype(&spec_page_reserve) reserve;
    decltype(&spec_page_fork) fork;
    decltype(&spec_page_release) release;
    decltype(&spec_page_compact) compact;
    decltype(&spec_page_copy) copy;
    decltype(&spec_rollback) rollback;
    decltype(&spec_cache_rollback) commit;
    PyObject *raw_stream;   // torch._C._cuda_getCurrentRawStream
} lib;

// The library's call without the interpreter's lock: a launch may wait for room in the stream's queue, and other
// threads go on meanwhile.  (The caller's frame keeps the tensors.)
template <typename F, typename... A>
sv_status unlocked(F call, A... args) {
    PyThreadState *const state = PyEval_SaveThread();
    const sv_status status = call(args...);
    PyEval_RestoreThread(state);
    return status;
}

struct Bad {};   // a Python error is set

[[noreturn]] void fail(const char *name, const char *format, ...) {
    char what[256];
    va_list a;
    va_start(a, format);
    vsnprintf(what, sizeof what, format, a);
    va_end(a);
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, what);
    throw Bad{};
}

constexpr auto I32 = c10::ScalarType::Int;
constexpr auto F32 = c10::ScalarType::Float;

// A tensor argument; the device of the first one seen is the call's.
struct Args {
    PyObject *const *v;
    int device = -1;

    const at::Tensor &tensor(int i, const char *name) {
        if (!THPVariable_Check(v[i])) fail(name, "a CUDA tensor");
        const at::Tensor &t = THPVariable_Unpack(v[i]);
        if (!t.is_cuda()) fail(name, "a CUDA tensor");
        const int d = t.get_device();
        if (device < 0) device = d;
        else if (device != d) fail(name, "on the other tensors' device");
        return t;
    }
    bool none(int i) const { return v[i] == Py_None; }
    long long whole(int i) const {
        const long long x = PyLong_AsLongLong(v[i]);
        if (x == -1 && PyErr_Occurred()) throw Bad{};
        return x;
    }
    int32_t i32(int i, const char *name) const {
        const long long x = whole(i);
        if (x < INT32_MIN || x > INT32_MAX) fail(name, "a 32-bit integer");
        return (int32_t)x;
    }
    float real(int i) const {
        const double x = PyFloat_AsDouble(v[i]);
        if (x == -1.0 && PyErr_Occurred()) throw Bad{};
        return (float)x;
    }
    // Pointer of a contiguous tensor of the given type, of `numel` elements unless negative.
    void *data(int i, const char *name, c10::ScalarType type, int64_t numel, int64_t *count = nullptr) {
        const at::Tensor &t = tensor(i, name);
        if (!t.is_contiguous()) fail(name, "contiguous");
        if (t.scalar_type() != type) fail(name, "%s, got %s", c10::toString(type), c10::toString(t.scalar_type()));
        if (numel >= 0 && t.numel() != numel) fail(name, "%lld elements, got %lld", (long long)numel, (long long)t.numel());
        if (count) *count = t.numel();
        return t.data_ptr();
    }
    void *optional(int i, const char *name, c10::ScalarType type, int64_t numel, int64_t *count = nullptr) {
        return none(i) ? nullptr : data(i, name, type, numel, count);
    }
    void *workspace(int i, size_t *bytes) {
        const at::Tensor &t = tensor(i, "workspace");
        if (!t.is_contiguous()) fail("workspace", "contiguous");
        *bytes = t.nbytes();
        if (*bytes < 256) fail("workspace", "256 bytes at least");
        return t.data_ptr();
    }
    // The stream argument: a raw handle, an object with .cuda_stream, or None (the current one).
    void *stream(int i) {
        PyObject *o = v[i];
        long long h;
        if (o == Py_None) {
            PyObject *d = PyLong_FromLong(device), *r = d ? PyObject_CallOneArg(lib.raw_stream, d) : nullptr;
            Py_XDECREF(d);
            if (!r) throw Bad{};
            h = PyLong_AsLongLong(r);
            Py_DECREF(r);
        } else if (PyLong_Check(o)) {
            h = PyLong_AsLongLong(o);
        } else {
            PyObject *r = PyObject_GetAttrString(o, "cuda_stream");
            if (!r) throw Bad{};
            h = PyLong_AsLongLong(r);
            Py_DECREF(r);
        }
        if (h == -1 && PyErr_Occurred()) throw Bad{};
        return reinterpret_cast<void *>(h);
    }
    // A [rows, heads, D] tensor, contiguous within a row; `stride` is the distance between rows.
    void *rows(int i, const char *name, c10::ScalarType type, int64_t R, int64_t heads, int64_t D, int64_t *stride) {
        const at::Tensor &t = tensor(i, name);
        if (t.scalar_type() != type) fail(name, "%s, got %s", c10::toString(type), c10::toString(t.scalar_type()));
        if (t.dim() != 3 || t.size(0) != R || t.size(1) != heads || t.size(2) != D)
            fail(name, "[%lld, %lld, %lld]", (long long)R, (long long)heads, (long long)D);
        if ((t.stride(2) != 1 && D != 1) || (t.stride(1) != D && heads != 1)) fail(name, "contiguous within a row");
        *stride = R > 1 ? t.stride(0) : heads * D;
        return t.data_ptr();
    }
    // k_cache, v_cache and block_table at i, i + 1, i + 2.
    sv_kv_cache cache(int i, int64_t B, c10::ScalarType *type) {
        const at::Tensor &k = tensor(i, "k_cache"), &v = tensor(i + 1, "v_cache");
        *type = k.scalar_type();
        if ((*type != c10::ScalarType::BFloat16 && *type != c10::ScalarType::Half) || v.scalar_type() != *type)
            fail("k_cache and v_cache", "both bfloat16 or both float16");
        if (k.dim() != 4 || k.sizes() != v.sizes() || k.strides() != v.strides())
            fail("k_cache and v_cache", "[pages, slots, heads, head_dim], of one shape and strides");
        if (k.stride(3) != 1) fail("k_cache and v_cache", "contiguous in head_dim");
        for (int d = 0; d < 4; d++)
            if (k.size(d) > INT32_MAX) fail("k_cache and v_cache", "smaller");
        const at::Tensor &t = tensor(i + 2, "block_table");
        if (t.scalar_type() != I32 || t.dim() != 2 || t.size(0) != B || !t.is_contiguous() || t.size(1) > INT32_MAX)
            fail("block_table", "contiguous int32 [%lld, max_pages]", (long long)B);
        sv_kv_cache c;
        c.k = k.data_ptr();
        c.v = v.data_ptr();
        c.page_stride = k.stride(0);
        c.token_stride = k.stride(1);
        c.head_stride = k.stride(2);
        c.num_pages = (int32_t)k.size(0);
        c.page_size = (int32_t)k.size(1);
        c.num_heads = (int32_t)k.size(2);
        c.head_dim = (int32_t)k.size(3);
        c.dtype = *type == c10::ScalarType::BFloat16 ? SV_BF16 : SV_F16;
        c.max_pages = (int32_t)t.size(1);
        c.block_table = static_cast<const int32_t *>(t.data_ptr());
        return c;
    }
};

int32_t count32(int64_t n, const char *name) {
    if (n > INT32_MAX) fail(name, "smaller");
    return (int32_t)n;
}
const int32_t *ints(void *p) { return static_cast<const int32_t *>(p); }

// q, k, v, q_weight, k_weight, eps, inv_freq, k_cache, v_cache, block_table, kv_seq_len, num_drafts,
// row_offsets, k_max, out_q, workspace, interleaved, rope_scale, stream
sv_status append(Args a) {
    int64_t n, half = 0, sq, sk, sv, so;
    size_t bytes;
    c10::ScalarType type;
    const int32_t *nd = ints(a.data(11, "num_drafts", I32, -1, &n));
    const sv_kv_cache c = a.cache(7, n, &type);
    const at::Tensor &q = a.tensor(0, "q");
    if (q.dim() != 3) fail("q", "[rows, heads, head_dim]");
    const int64_t R = q.size(0), Hq = q.size(1), D = c.head_dim;
    void *pq = a.rows(0, "q", type, R, Hq, D, &sq), *pk = a.rows(1, "k", type, R, c.num_heads, D, &sk),
         *pv = a.rows(2, "v", type, R, c.num_heads, D, &sv), *po = a.rows(14, "out_q", type, R, Hq, D, &so);
    void *qw = a.optional(3, "q_weight", type, D), *kw = a.optional(4, "k_weight", type, D);
    void *inv = a.optional(6, "inv_freq", F32, -1, &half);
    const int32_t *ro = ints(a.optional(12, "row_offsets", I32, n + 1)), *ln = ints(a.data(10, "kv_seq_len", I32, n));
    void *ws = a.workspace(15, &bytes);
    const int il = PyObject_IsTrue(a.v[16]);
    if (il < 0) throw Bad{};
    return unlocked(lib.append, pq, pk, pv, sq, sk, sv, count32(Hq, "q"), qw, kw, a.real(5), static_cast<const float *>(inv),
                      count32(2 * half, "inv_freq"), il, a.real(17), nd, ro, ln, count32(n, "num_drafts"),
                      a.i32(13, "k_max"), count32(R, "q"), c, po, so, ws, a.stream(18));
}

// q, k_cache, v_cache, block_table, kv_seq_len, num_drafts, row_offsets, k_max, scale, window, sinks, out,
// out_lse, workspace, stream
sv_status attention(Args a) {
    int64_t n, sq;
    size_t bytes;
    c10::ScalarType type;
    const int32_t *nd = ints(a.data(5, "num_drafts", I32, -1, &n));
    const sv_kv_cache c = a.cache(1, n, &type);
    const at::Tensor &q = a.tensor(0, "q");
    if (q.dim() != 3) fail("q", "[rows, heads, head_dim]");
    const int64_t R = q.size(0), Hq = q.size(1);
    void *pq = a.rows(0, "q", type, R, Hq, c.head_dim, &sq);
    const int32_t *ro = ints(a.optional(6, "row_offsets", I32, n + 1)), *ln = ints(a.data(4, "kv_seq_len", I32, n));
    void *out = a.data(11, "out", type, R * Hq * c.head_dim), *lse = a.optional(12, "out_lse", F32, R * Hq);
    void *ws = a.workspace(13, &bytes);
    return unlocked(lib.attention, pq, sq, count32(Hq, "q"), nd, ro, ln, count32(n, "num_drafts"), a.i32(7, "k_max"),
                         count32(R, "q"), c, a.real(8), a.i32(9, "window"), a.i32(10, "sinks"), out,
                         static_cast<float *>(lse), ws, bytes, a.stream(14));
}

struct State {
    int32_t *len, *table, *ref;
    int32_t B, max_pages, num_pages;
};
// kv_seq_len (if any), block_table and ref_count at i - 1, i, i + 1.
State state(Args &a, int i, bool with_len) {
    const at::Tensor &t = a.tensor(i, "block_table");
    if (t.dim() != 2) fail("block_table", "[B, max_pages]");
    State s;
    int64_t pages;
    s.table = static_cast<int32_t *>(a.data(i, "block_table", I32, -1));
    s.B = count32(t.size(0), "block_table");
    s.max_pages = count32(t.size(1), "block_table");
    s.len = with_len ? static_cast<int32_t *>(a.data(i - 1, "kv_seq_len", I32, s.B)) : nullptr;
    s.ref = static_cast<int32_t *>(a.data(i + 1, "ref_count", I32, -1, &pages));
    s.num_pages = count32(pages, "ref_count");
    return s;
}

// num_drafts, kv_seq_len, block_table, ref_count, page_size, workspace, stream
sv_status reserve(Args a) {
    size_t bytes;
    const State s = state(a, 2, true);
    const int32_t *nd = ints(a.data(0, "num_drafts", I32, s.B));
    void *ws = a.workspace(5, &bytes);
    return unlocked(lib.reserve, nd, s.len, s.B, s.table, s.max_pages, s.ref, s.num_pages, a.i32(4, "page_size"), ws, bytes,
                       a.stream(6));
}

// parents, children, fork_len, kv_seq_len, block_table, ref_count, page_size, copy_src, copy_dst, workspace, stream
sv_status fork(Args a) {
    int64_t n;
    size_t bytes;
    const State s = state(a, 4, true);
    const int32_t *pa = ints(a.data(0, "parents", I32, -1, &n)), *ch = ints(a.data(1, "children", I32, n)),
                  *fl = ints(a.optional(2, "fork_len", I32, n));
    int32_t *src = static_cast<int32_t *>(a.data(7, "copy_src", I32, n)), *dst = static_cast<int32_t *>(a.data(8, "copy_dst", I32, n));
    void *ws = a.workspace(9, &bytes);
    return unlocked(lib.fork, pa, ch, fl, count32(n, "parents"), s.len, s.B, s.table, s.max_pages, s.ref, s.num_pages,
                    a.i32(6, "page_size"), src, dst, ws, bytes, a.stream(10));
}

// kv_seq_len, block_table, ref_count, page_size, window, sinks, workspace, stream
sv_status release(Args a) {
    size_t bytes;
    const State s = state(a, 1, true);
    void *ws = a.workspace(6, &bytes);
    return unlocked(lib.release, s.len, s.B, s.table, s.max_pages, s.ref, s.num_pages, a.i32(3, "page_size"), a.i32(4, "window"),
                       a.i32(5, "sinks"), ws, a.stream(7));
}

// block_table, ref_count, copy_src, copy_dst, workspace, stream
sv_status compact(Args a) {
    int64_t cap;
    size_t bytes;
    const State s = state(a, 0, false);
    int32_t *src = static_cast<int32_t *>(a.data(2, "copy_src", I32, -1, &cap)), *dst = static_cast<int32_t *>(a.data(3, "copy_dst", I32, cap));
    void *ws = a.workspace(4, &bytes);
    return unlocked(lib.compact, s.B, s.table, s.max_pages, s.ref, s.num_pages, src, dst, count32(cap, "copy_src"), ws, bytes,
                       a.stream(5));
}

// k_cache, v_cache, copy_src, copy_dst, workspace, stream
sv_status copy(Args a) {
    const at::Tensor &k = a.tensor(0, "k_cache");
    const int dims = (int)k.dim();
    if (dims < 2 || dims > 5) fail("k_cache", "[pages, ...] or [layers, pages, slots, heads, head_dim]");
    void *pv = nullptr;
    if (!a.none(1)) {
        const at::Tensor &v = a.tensor(1, "v_cache");
        if (v.sizes() != k.sizes() || v.strides() != k.strides() || v.scalar_type() != k.scalar_type())
            fail("v_cache", "like k_cache");
        pv = v.data_ptr();
    }
    // a page's dimensions have to fill it without gaps, in any order
    const int page_dim = dims == 5 ? 1 : 0;
    int64_t dense = 1;
    bool used[5] = {};
    for (int step = page_dim + 1; step < dims; step++)
        for (int d = page_dim + 1; d < dims; d++)
            if (!used[d] && (k.stride(d) == dense || k.size(d) == 1)) {
                used[d] = true;
                dense *= k.size(d);
            }
    for (int d = page_dim + 1; d < dims; d++)
        if (!used[d]) fail("k_cache", "contiguous within a page");
    const int64_t size = k.element_size();
    int64_t n;
    size_t bytes;
    const int32_t *src = ints(a.data(2, "copy_src", I32, -1, &n)), *dst = ints(a.data(3, "copy_dst", I32, n));
    void *ws = a.workspace(4, &bytes);
    return unlocked(lib.copy, k.data_ptr(), pv, dense * size, k.stride(page_dim) * size, page_dim ? count32(k.size(0), "k_cache") : 1,
                    page_dim ? k.stride(0) * size : 0, count32(k.size(page_dim), "k_cache"), src, dst,
                    count32(n, "copy_src"), ws, a.stream(5));
}

// kv_seq_len, accept_len, num_drafts, workspace, stream.  The package's spec_rollback, with the checks that it has in
// Python: tensors may be on any device, a workspace of any size, and the library refuses what is None.
sv_status rollback(Args a) {
    int64_t n;
    int32_t *ln = static_cast<int32_t *>(a.data(0, "kv_seq_len", I32, -1, &n));
    const int device = a.device;
    auto any = [&](int i, const char *name, bool counted) -> void * {
        a.device = -1;
        if (a.none(i)) return nullptr;
        if (counted) return a.data(i, name, I32, n);
        const at::Tensor &t = a.tensor(i, name);
        if (!t.is_contiguous()) fail(name, "contiguous");
        return t.data_ptr();
    };
    const int32_t *acc = ints(any(1, "accept_len", true)), *nd = ints(any(2, "num_drafts", true));
    void *ws = any(3, "workspace", false);
    a.device = device;
    return unlocked(lib.rollback, ln, acc, nd, count32(n, "kv_seq_len"), ws, a.stream(4));
}

// kv_seq_len, accept_len, num_drafts, workspace, stream
sv_status commit(Args a) {
    int64_t n;
    size_t bytes;
    int32_t *ln = static_cast<int32_t *>(a.data(0, "kv_seq_len", I32, -1, &n));
    const int32_t *acc = ints(a.data(1, "accept_len", I32, n)), *nd = ints(a.data(2, "num_drafts", I32, n));
    void *ws = a.workspace(3, &bytes);
    return unlocked(lib.commit, ln, acc, nd, count32(n, "kv_seq_len"), ws, a.stream(4));
}

template <sv_status (*F)(Args), int N>
PyObject *call(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
        return nullptr;
    }
    if (!lib.raw_stream) {
        PyErr_SetString(PyExc_RuntimeError, "init() has not been called");
        return nullptr;
    }
    try {
        return PyLong_FromLong((long)F(Args{v}));
    } catch (const Bad &) {
        return nullptr;
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// Addresses of the entry points in the order of Entry, then the raw-stream function.
PyObject *init(PyObject *, PyObject *const *v, Py_ssize_t n) {
    if (n != 10) {
        PyErr_SetString(PyExc_TypeError, "expected 10 arguments");
        return nullptr;
    }
    void *p[9];
    for (int i = 0; i < 9; i++) {
        p[i] = PyLong_AsVoidPtr(v[i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null entry point");
            return nullptr;
        }
    }
    lib.append = reinterpret_cast<decltype(lib.append)>(p[0]);
    lib.attention = reinterpret_cast<decltype(lib.attention)>(p[1]);
    lib.reserve = reinterpret_cast<decltype(lib.reserve)>(p[2]);
    lib.fork = reinterpret_cast<decltype(lib.fork)>(p[3]);
    lib.release = reinterpret_cast<decltype(lib.release)>(p[4]);
    lib.compact = reinterpret_cast<decltype(lib.compact)>(p[5]);
    lib.copy = reinterpret_cast<decltype(lib.copy)>(p[6]);
    lib.rollback = reinterpret_cast<decltype(lib.rollback)>(p[7]);
    lib.commit = reinterpret_cast<decltype(lib.commit)>(p[8]);
    Py_INCREF(v[9]);
    lib.raw_stream = v[9];
    Py_RETURN_NONE;
}

#define FAST(name, f) {name, (PyCFunction)(void (*)(void))(f), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("init", init),
                         FAST("append", (call<append, 19>)),
                         FAST("attention", (call<attention, 15>)),
                         FAST("reserve", (call<reserve, 7>)),
                         FAST("fork", (call<fork, 11>)),
                         FAST("release", (call<release, 8>)),
                         FAST("compact", (call<compact, 6>)),
                         FAST("copy", (call<copy, 6>)),
                         FAST("rollback", (call<rollback, 5>)),
                         FAST("commit", (call<commit, 5>)),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Checks of tensors before the cache-side calls.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
