// kvattend_py.cpp - Python binding of the operators of kvattend.h: reads
// torch tensors' addresses and strides, checks them, and calls the C entry
// points of libkvcodec.so.
//
// A decoding step makes these calls with a few microseconds of GPU work each,
// so what a call costs on the host counts: the same marshalling through ctypes
// took 6 to 12 us a call, here it is 1 to 2 us besides the launches.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "kvattend.h"

namespace {

// The entry points, of the library that kvcodec loaded.
decltype(&kvc_norm_rotate) f_norm_rotate = nullptr;
decltype(&kvpage_write) f_page_write = nullptr;
decltype(&kvpage_read) f_page_read = nullptr;
decltype(&kvpage_attend) f_page_attend = nullptr;
decltype(&kvpool_attend) f_pool_attend = nullptr;
decltype(&kvpage_append) f_page_append = nullptr;
decltype(&kvpage_attend_window) f_page_attend_window = nullptr;
decltype(&kvpage_attend_prompt) f_page_attend_prompt = nullptr;

PyObject* g_kvc_error = nullptr;   // kvcodec.KvcError
PyObject* g_raw_stream = nullptr;  // device -> handle of its current stream
PyObject* g_device = nullptr;      // the current device
PyObject* g_device_guard = nullptr;  // torch.cuda.device
PyObject* g_as_floats = nullptr;   // any sequence -> contiguous float32 array

// A refused argument: the Python error is set.
struct Refused {};

[[noreturn]] void refuse(const std::string& what) {
    PyErr_SetString(PyExc_ValueError, what.c_str());
    throw Refused{};
}
void py_ok(bool ok) {
    if (!ok) throw Refused{};
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

// The arguments of a call by name; `given` holds NULL for what was left out or None.
template <int N>
struct Args {
    PyObject* given[N] = {};
    const at::Tensor* seen[N + 4] = {};
    int n_seen = 0;

    Args(const char* function, const char* const (&names)[N], int positional, int required, PyObject* const* args,
         Py_ssize_t nargs, PyObject* kwnames) {
        if (nargs > positional) {
            PyErr_Format(PyExc_TypeError, "%s: takes at most %d positional arguments", function, positional);
            throw Refused{};
        }
        for (Py_ssize_t i = 0; i < nargs; ++i) given[i] = args[i];
        const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < nk; ++k) {
            PyObject* key = PyTuple_GET_ITEM(kwnames, k);
            int at = -1;
            for (int i = 0; i < N && at < 0; ++i)
                if (PyUnicode_CompareWithASCIIString(key, names[i]) == 0) at = i;
            if (at < 0 || given[at]) {
                PyErr_Format(PyExc_TypeError, "%s: unexpected or repeated argument %U", function, key);
                throw Refused{};
            }
            given[at] = args[nargs + k];
        }
        for (int i = 0; i < required; ++i)
            if (!given[i]) {
                PyErr_Format(PyExc_TypeError, "%s: missing argument %s", function, names[i]);
                throw Refused{};
            }
        for (int i = 0; i < N; ++i)
            if (given[i] == Py_None) given[i] = nullptr;
    }

    const at::Tensor* tensor(PyObject* o, const char* what) {
        if (!o) return nullptr;
        if (!THPVariable_Check(o)) refuse(std::string(what) + ": expected a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        if (t.layout() != at::kStrided) refuse(std::string(what) + ": expected a strided tensor");
        seen[n_seen++] = &t;
        return &t;
    }
    const at::Tensor& need(PyObject* o, const char* what) {
        const at::Tensor* t = tensor(o, what);
        if (!t) refuse(std::string(what) + ": tensor required");
        return *t;
    }
};

void want_type(const at::Tensor& t, at::ScalarType type, const char* what) {
    if (t.scalar_type() != type)
        refuse(std::string(what) + ": expected " + at::toString(type) + ", got " + at::toString(t.scalar_type()));
}
void want_shape(const at::Tensor& t, at::IntArrayRef shape, const char* what) {
    if (t.sizes() != shape) refuse(std::string(what) + ": expected shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}

// bf16 rows [n][heads][d]; strides of dimensions of size 1 are not used.
kvc_rows rows_of(const at::Tensor& t, at::IntArrayRef shape, const char* what) {
    want_type(t, at::kBFloat16, what);
    want_shape(t, shape, what);
    const auto s = t.strides();
    if (s[2] != 1 && shape[0]) refuse(std::string(what) + ": the last dimension must be contiguous");
    return kvc_rows{t.data_ptr(), (uint64_t)s[0], (uint64_t)s[1]};
}
// A contiguous tensor of this type and shape.
void* plain(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape, const char* what) {
    want_type(t, type, what);
    want_shape(t, shape, what);
    if (!t.is_contiguous()) refuse(std::string(what) + ": expected a contiguous tensor");
    return t.data_ptr();
}
void* bytes_of(const at::Tensor& t, const char* what) {
    if (t.scalar_type() != at::kByte || !t.is_contiguous()) refuse(std::string(what) + ": expected a contiguous uint8 tensor");
    return t.data_ptr();
}

// N uint32 values from a tuple or list, or the bytes of a ctypes structure of them.
template <int N>
void words(PyObject* o, uint32_t (&w)[N], const char* what) {
    if (PyTuple_Check(o) || PyList_Check(o)) {
        if (PySequence_Fast_GET_SIZE(o) != N) refuse(std::string(what) + ": expected " + std::to_string(N) + " numbers");
        for (int i = 0; i < N; ++i) {
            const long long v = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(o, i));
            py_ok(!(v == -1 && PyErr_Occurred()));
            if (v < 0 || v > 0xFFFFFFFFll) refuse(std::string(what) + ": number out of range");
            w[i] = (uint32_t)v;
        }
        return;
    }
    Py_buffer b;
    py_ok(PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) == 0);
    const bool ok = b.len == (Py_ssize_t)sizeof(w);
    if (ok) memcpy(w, b.buf, sizeof(w));
    PyBuffer_Release(&b);
    if (!ok) refuse(std::string(what) + ": expected " + std::to_string(N) + " numbers");
}
kvc_pages spec_of(PyObject* o) {
    uint32_t w[5];
    words(o, w, "spec");
    return kvc_pages{w[0], w[1], w[2], w[3], w[4]};
}
kvc_shape shape_of(PyObject* o) {
    if (PyTuple_Check(o) || PyList_Check(o) || PyObject_CheckBuffer(o)) {
        uint32_t w[4];
        words(o, w, "shape");
        return kvc_shape{w[0], w[1], w[2], w[3]};
    }
    PyObject* t = PySequence_Tuple(o);
    py_ok(t != nullptr);
    uint32_t w[4];
    try {
        words(t, w, "shape");
    } catch (...) {
        Py_DECREF(t);
        throw;
    }
    Py_DECREF(t);
    return kvc_shape{w[0], w[1], w[2], w[3]};
}

uint32_t whole(PyObject* o, const char* what) {
    const long long v = PyLong_AsLongLong(o);
    py_ok(!(v == -1 && PyErr_Occurred()));
    if (v < 0 || v > 0xFFFFFFFFll) refuse(std::string(what) + ": number out of range");
    return (uint32_t)v;
}
float number(PyObject* o, float otherwise) {
    if (!o) return otherwise;
    const double v = PyFloat_AsDouble(o);
    py_ok(!(v == -1.0 && PyErr_Occurred()));
    return (float)v;
}
uint32_t count32(int64_t n, const char* what) {
    if (n > 0x7FFFFFFFll) refuse(std::string(what) + ": too many elements");
    return (uint32_t)n;
}

long long call_int(PyObject* f, PyObject* arg) {
    PyObject* r = arg ? PyObject_CallOneArg(f, arg) : PyObject_CallNoArgs(f);
    py_ok(r != nullptr);
    const long long v = (long long)PyLong_AsUnsignedLongLongMask(r);
    Py_DECREF(r);
    py_ok(!PyErr_Occurred());
    return v;
}

// call(stream) with the tensors' device current and the stream given, or that device's current one.
template <class A, class F>
PyObject* launch(const char* what, A& a, PyObject* stream, F call) {
    const at::Device device = a.seen[0]->device();
    for (int i = 1; i < a.n_seen; ++i)
        if (a.seen[i]->device() != device) refuse(std::string(what) + ": tensors are on different devices");
    if (!device.is_cuda()) refuse("expected a GPU tensor");
    PyObject* index = PyLong_FromLong(device.index());
    py_ok(index != nullptr);
    PyObject* guard = nullptr;
    int rc = 0;
    bool ok = true;
    try {
        if (call_int(g_device, nullptr) != device.index()) {
            guard = PyObject_CallOneArg(g_device_guard, index);
            py_ok(guard != nullptr);
            PyObject* in = PyObject_CallMethod(guard, "__enter__", nullptr);
            if (!in) Py_CLEAR(guard);
            py_ok(in != nullptr);
            Py_DECREF(in);
        }
        long long handle;
        if (!stream) {
            handle = call_int(g_raw_stream, index);
        } else if (PyLong_Check(stream)) {
            handle = (long long)PyLong_AsUnsignedLongLongMask(stream);
        } else {
            PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
            py_ok(h != nullptr);
            handle = (long long)PyLong_AsUnsignedLongLongMask(h);
            Py_DECREF(h);
        }
        py_ok(!PyErr_Occurred());
        Py_BEGIN_ALLOW_THREADS;
        rc = call(reinterpret_cast<hipStream_t>(handle));
        Py_END_ALLOW_THREADS;
    } catch (const Refused&) {
        ok = false;
    }
    Py_DECREF(index);
    if (guard) {
        PyObject *type, *value, *trace;
        PyErr_Fetch(&type, &value, &trace);
        PyObject* out = PyObject_CallMethod(guard, "__exit__", "OOO", Py_None, Py_None, Py_None);
        Py_XDECREF(out);
        if (type) PyErr_Restore(type, value, trace);
        Py_DECREF(guard);
        if (!out) ok = false;
    }
    if (!ok) return nullptr;
    if (rc != KVC_OK) {
        PyObject* e = PyObject_CallFunction(g_kvc_error, "is", rc, what);
        if (e) PyErr_SetObject(g_kvc_error, e);
        Py_XDECREF(e);
        return nullptr;
    }
    Py_RETURN_NONE;
}

// Python errors for whatever a call throws.
template <class F>
PyObject* guarded(F f) {
    try {
        return f();
    } catch (const Refused&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// Host floats: the buffer of a contiguous float32 array, else a copy of one.
struct Floats {
    Py_buffer b{};
    bool held = false;
    explicit Floats(PyObject* o) {
        take(o);
        if (held && !fits()) release();
        if (!held) {
            PyErr_Clear();
            PyObject* a = PyObject_CallOneArg(g_as_floats, o);
            py_ok(a != nullptr);
            take(a);
            Py_DECREF(a);  // the buffer holds it
            py_ok(held);
        }
    }
    ~Floats() { release(); }
    void take(PyObject* o) { held = PyObject_GetBuffer(o, &b, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) == 0; }
    bool fits() const { return b.itemsize == 4 && b.format && b.format[0] == 'f' && b.format[1] == 0; }
    void release() {
        if (held) PyBuffer_Release(&b);
        held = false;
    }
    const float* data() const { return static_cast<const float*>(b.buf); }
    uint32_t size() const { return (uint32_t)(b.len / 4); }
};

const char kRotateDoc[] =
    "kvc_norm_rotate(q, k, positions, inv_freq, q_out, k_out, q_weight=None, k_weight=None, eps=1e-6, pairing=0,\n"
    "                stream=None)\n\n"
    "q, q_out: rows [n, q_heads, d]; k, k_out: rows [n, kv_heads, d] (either pair may be None); the same tensor\n"
    "for in place. positions: int64 [n]; inv_freq: host floats, one for each pair that is turned (empty: none);\n"
    "q_weight, k_weight: bf16 [d] or None (no norm).";
PyObject* norm_rotate(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const names[11] = {"q", "k", "positions", "inv_freq", "q_out", "k_out", "q_weight", "k_weight",
                                              "eps", "pairing", "stream"};
        Args<11> a("kvc_norm_rotate", names, 11, 6, args, nargs, kwnames);
        PyObject** g = a.given;
        if ((!g[0]) != (!g[4]) || (!g[1]) != (!g[5])) refuse("each input needs its output");
        const at::Tensor& first = a.need(g[0] ? g[0] : g[1], "q or k");
        if (first.dim() != 3) refuse("expected rows [tokens, heads, head_dim]");
        const int64_t n = first.size(0), d = first.size(2);
        kvc_rows in[2] = {}, out[2] = {};
        int64_t heads[2] = {};
        const void* weight[2] = {};
        static const char* const what[2][3] = {{"q", "q_out", "q_weight"}, {"k", "k_out", "k_weight"}};
        for (int i = 0; i < 2; ++i) {
            if (!g[i]) continue;
            const at::Tensor& x = a.need(g[i], what[i][0]);
            if (x.dim() != 3) refuse("expected rows [tokens, heads, head_dim]");
            heads[i] = x.size(1);
            in[i] = rows_of(x, {n, heads[i], d}, what[i][0]);
            out[i] = rows_of(a.need(g[4 + i], what[i][1]), {n, heads[i], d}, what[i][1]);
            if (g[6 + i]) weight[i] = plain(a.need(g[6 + i], what[i][2]), at::kBFloat16, {d}, what[i][2]);
        }
        if (!g[3]) refuse("inv_freq: floats required");
        const Floats f(g[3]);
        const void* at = nullptr;
        if (g[2])
            at = plain(a.need(g[2], "positions"), at::kLong, {n}, "positions");
        else if (f.size())
            refuse("positions: tensor required");
        const float eps = number(g[8], 1e-6f);
        const uint32_t pairing = g[9] ? whole(g[9], "pairing") : 0, nt = count32(n, "tokens"),
                       hq = count32(heads[0], "q_heads"), hk = count32(heads[1], "kv_heads"), dd = count32(d, "head_dim");
        return launch("kvc_norm_rotate", a, g[10], [&](hipStream_t s) {
            return f_norm_rotate(nt, hq, hk, dd, g[0] ? &in[0] : nullptr, g[1] ? &in[1] : nullptr, weight[0], weight[1],
                                   eps, static_cast<const int64_t*>(at), f.size() ? f.data() : nullptr, f.size(), pairing,
                                   g[0] ? &out[0] : nullptr, g[1] ? &out[1] : nullptr, s);
        });
    });
}

const char kWriteDoc[] =
    "kvpage_write(spec, pages, k, v, slots, dev_status=None, stream=None)\n\n"
    "k, v: rows [n, num_kv_heads, head_dim]; slots: int64 [n], page * page_tokens + offset (negative: skipped);\n"
    "dev_status: int32 [1] or None.";
const char kReadDoc[] =
    "kvpage_read(spec, pages, slots, k_out, v_out, dev_status=None, stream=None)\n\n"
    "The tokens of `slots` into rows k_out, v_out (rows of negative slots are left as they were).";
template <bool WRITE>
PyObject* page_copy(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const wn[7] = {"spec", "pages", "k", "v", "slots", "dev_status", "stream"};
        static const char* const rn[7] = {"spec", "pages", "slots", "k_out", "v_out", "dev_status", "stream"};
        const char* const what = WRITE ? "kvpage_write" : "kvpage_read";
        Args<7> a(what, WRITE ? wn : rn, 7, 5, args, nargs, kwnames);
        PyObject** g = a.given;
        if (!g[0]) refuse("spec: description required");
        const kvc_pages spec = spec_of(g[0]);
        const at::Tensor& pages = a.need(g[1], "pages");
        const at::Tensor& slots = a.need(g[WRITE ? 4 : 2], "slots");
        const int64_t n = slots.numel();
        const int64_t shape[3] = {n, spec.num_kv_heads, spec.head_dim};
        void* at = bytes_of(pages, "pages");
        const kvc_rows k = rows_of(a.need(g[WRITE ? 2 : 3], "k"), shape, "k"), v = rows_of(a.need(g[WRITE ? 3 : 4], "v"), shape, "v");
        const auto* sl = static_cast<const int64_t*>(plain(slots, at::kLong, {n}, "slots"));
        int32_t* st = g[5] ? static_cast<int32_t*>(plain(a.need(g[5], "dev_status"), at::kInt, {1}, "dev_status")) : nullptr;
        const uint32_t nt = count32(n, "slots");
        const size_t size = (size_t)pages.numel();
        return launch(what, a, g[6], [&](hipStream_t s) {
            return WRITE ? f_page_write(&spec, at, size, nt, &k, &v, sl, st, s) : f_page_read(&spec, at, size, nt, sl, &k, &v, st, s);
        });
    });
}

const char kAppendDoc[] =
    "kvpage_append(spec, pages, q, k, v, positions, inv_freq, slots, q_out, q_weight=None, k_weight=None, eps=1e-6,\n"
    "              pairing=0, dev_status=None, stream=None)\n\n"
    "q, q_out: rows [n, q_heads, head_dim] (both may be None; the same tensor for in place); k, v: rows\n"
    "[n, num_kv_heads, head_dim]; positions, inv_freq and weights as for kvc_norm_rotate, slots as for kvpage_write.";
PyObject* page_append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const names[15] = {"spec", "pages", "q", "k", "v", "positions", "inv_freq", "slots", "q_out",
                                              "q_weight", "k_weight", "eps", "pairing", "dev_status", "stream"};
        Args<15> a("kvpage_append", names, 15, 9, args, nargs, kwnames);
        PyObject** g = a.given;
        if (!g[0]) refuse("spec: description required");
        if ((!g[2]) != (!g[8])) refuse("q needs q_out");
        const kvc_pages spec = spec_of(g[0]);
        const at::Tensor& pages = a.need(g[1], "pages");
        void* at = bytes_of(pages, "pages");
        const at::Tensor& slots = a.need(g[7], "slots");
        const int64_t n = slots.numel(), d = spec.head_dim;
        const int64_t shape[3] = {n, spec.num_kv_heads, d};
        const kvc_rows k = rows_of(a.need(g[3], "k"), shape, "k"), v = rows_of(a.need(g[4], "v"), shape, "v");
        const auto* sl = static_cast<const int64_t*>(plain(slots, at::kLong, {n}, "slots"));
        kvc_rows q{}, out{};
        int64_t heads = 0;
        if (g[2]) {
            const at::Tensor& x = a.need(g[2], "q");
            if (x.dim() != 3) refuse("q: expected rows [tokens, heads, head_dim]");
            heads = x.size(1);
            q = rows_of(x, {n, heads, d}, "q");
            out = rows_of(a.need(g[8], "q_out"), {n, heads, d}, "q_out");
        }
        const void* weight[2] = {};
        static const char* const what[2] = {"q_weight", "k_weight"};
        for (int i = 0; i < 2; ++i)
            if (g[9 + i]) weight[i] = plain(a.need(g[9 + i], what[i]), at::kBFloat16, {d}, what[i]);
        if (!g[6]) refuse("inv_freq: floats required");
        const Floats f(g[6]);
        const void* pos = nullptr;
        if (g[5])
            pos = plain(a.need(g[5], "positions"), at::kLong, {n}, "positions");
        else if (f.size())
            refuse("positions: tensor required");
        const float eps = number(g[11], 1e-6f);
        const uint32_t pairing = g[12] ? whole(g[12], "pairing") : 0, nt = count32(n, "slots"), hq = count32(heads, "q_heads");
        int32_t* st = g[13] ? static_cast<int32_t*>(plain(a.need(g[13], "dev_status"), at::kInt, {1}, "dev_status")) : nullptr;
        const size_t size = (size_t)pages.numel();
        return launch("kvpage_append", a, g[14], [&](hipStream_t s) {
            return f_page_append(&spec, at, size, nt, hq, g[2] ? &q : nullptr, &k, &v, weight[0], weight[1], eps,
                                 static_cast<const int64_t*>(pos), f.size() ? f.data() : nullptr, f.size(), pairing, sl,
                                 g[2] ? &out : nullptr, st, s);
        });
    });
}

// What the attention calls have in common.
struct Attend {
    uint32_t n, hq;
    int64_t d;
    kvc_rows q, out;
    float* lse = nullptr;
    float scale;
    void* ws;
    size_t ws_bytes;
    int32_t* status = nullptr;
    template <class A>
    Attend(A& a, uint32_t head_dim, PyObject* qo, PyObject* oo, PyObject* wo, PyObject* lo, PyObject* so, PyObject* to) {
        const at::Tensor& t = a.need(qo, "q");
        if (t.dim() != 3) refuse("q: expected rows [sequences, heads, head_dim]");
        d = t.size(2);
        if (d != head_dim) refuse("q: expected head_dim " + std::to_string(head_dim) + ", got " + std::to_string(d));
        n = count32(t.size(0), "q");
        hq = count32(t.size(1), "q");
        q = rows_of(t, t.sizes(), "q");
        out = rows_of(a.need(oo, "out"), t.sizes(), "out");
        const at::Tensor& w = a.need(wo, "ws");
        ws = bytes_of(w, "ws");
        ws_bytes = (size_t)w.numel();
        if (lo) lse = static_cast<float*>(plain(a.need(lo, "lse"), at::kFloat, {t.size(0), t.size(1)}, "lse"));
        scale = number(so, 1.0f / std::sqrt((float)d));
        if (to) status = static_cast<int32_t*>(plain(a.need(to, "dev_status"), at::kInt, {1}, "dev_status"));
    }
};
struct Table {
    const int32_t *table, *lens;
    uint32_t cols;
    uint64_t stride;
    template <class A>
    Table(A& a, PyObject* to, PyObject* lo, int64_t n) {
        const at::Tensor& t = a.need(to, "table");
        if (t.scalar_type() != at::kInt || t.dim() != 2 || t.size(0) != n || (n && t.size(1) > 1 && t.stride(1) != 1))
            refuse("table: expected int32 [" + std::to_string(n) + ", columns] with contiguous rows");
        table = static_cast<const int32_t*>(t.data_ptr());
        cols = count32(t.size(1), "table");
        stride = (uint64_t)t.stride(0);
        lens = static_cast<const int32_t*>(plain(a.need(lo, "lens"), at::kInt, {(int64_t)n}, "lens"));
    }
};

const char kPageDoc[] =
    "kvpage_attend(spec, pages, q, table, lens, out, ws, lse=None, scale=None, dev_status=None, stream=None)\n\n"
    "q, out: rows [n, q_heads, head_dim]; table: int32 [n, columns] page numbers; lens: int32 [n]; ws: uint8\n"
    "workspace (kvpage_attend_workspace_bytes of columns * page_tokens); lse: float32 [n, q_heads] or None;\n"
    "scale: 1 / sqrt(head_dim) if None.";
PyObject* page_attend(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const names[11] = {"spec", "pages", "q", "table", "lens", "out", "ws", "lse", "scale", "dev_status",
                                              "stream"};
        Args<11> a("kvpage_attend", names, 11, 7, args, nargs, kwnames);
        PyObject** g = a.given;
        if (!g[0]) refuse("spec: description required");
        const kvc_pages spec = spec_of(g[0]);
        const at::Tensor& pages = a.need(g[1], "pages");
        void* at = bytes_of(pages, "pages");
        const Attend x(a, spec.head_dim, g[2], g[5], g[6], g[7], g[8], g[9]);
        const Table t(a, g[3], g[4], x.n);
        const size_t size = (size_t)pages.numel();
        return launch("kvpage_attend", a, g[10], [&](hipStream_t s) {
            return f_page_attend(&spec, at, size, x.n, x.hq, &x.q, t.table, t.cols, t.stride, t.lens, x.scale, &x.out, x.lse,
                                 x.ws, x.ws_bytes, x.status, s);
        });
    });
}

const char kWindowDoc[] =
    "kvpage_attend_window(spec, pages, q, table, lens, window, sinks, out, ws, lse=None, scale=None, dev_status=None,\n"
    "                     stream=None)\n\n"
    "kvpage_attend of the last `window` tokens (0: all) and the first `sinks`; ws: uint8 workspace\n"
    "(kvpage_attend_window_workspace_bytes).";
PyObject* page_attend_window(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const names[13] = {"spec", "pages", "q", "table", "lens", "window", "sinks", "out", "ws", "lse",
                                              "scale", "dev_status", "stream"};
        Args<13> a("kvpage_attend_window", names, 13, 9, args, nargs, kwnames);
        PyObject** g = a.given;
        if (!g[0] || !g[5] || !g[6]) refuse("spec, window and sinks are required");
        const kvc_pages spec = spec_of(g[0]);
        const at::Tensor& pages = a.need(g[1], "pages");
        void* at = bytes_of(pages, "pages");
        const uint32_t window = whole(g[5], "window"), sinks = whole(g[6], "sinks");
        const Attend x(a, spec.head_dim, g[2], g[7], g[8], g[9], g[10], g[11]);
        const Table t(a, g[3], g[4], x.n);
        const size_t size = (size_t)pages.numel();
        return launch("kvpage_attend_window", a, g[12], [&](hipStream_t s) {
            return f_page_attend_window(&spec, at, size, x.n, x.hq, &x.q, t.table, t.cols, t.stride, t.lens, window, sinks,
                                        x.scale, &x.out, x.lse, x.ws, x.ws_bytes, x.status, s);
        });
    });
}

const char kPromptDoc[] =
    "kvpage_attend_prompt(spec, pages, q, starts, table, lens, out, ws, window=0, sinks=0, lse=None, scale=None,\n"
    "                     dev_status=None, stream=None)\n\n"
    "q, out: rows [n, q_heads, head_dim] of the new tokens of all sequences; starts: int32 [sequences + 1], first row\n"
    "of each and the end of the last; table: int32 [sequences, columns]; lens: int32 [sequences], the new tokens\n"
    "among them; ws: uint8 workspace (kvpage_attend_prompt_workspace_bytes); lse: float32 [n, q_heads] or None.";
PyObject* page_attend_prompt(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const names[14] = {"spec", "pages", "q", "starts", "table", "lens", "out", "ws", "window", "sinks",
                                              "lse", "scale", "dev_status", "stream"};
        Args<14> a("kvpage_attend_prompt", names, 14, 8, args, nargs, kwnames);
        PyObject** g = a.given;
        if (!g[0]) refuse("spec: description required");
        const kvc_pages spec = spec_of(g[0]);
        const at::Tensor& pages = a.need(g[1], "pages");
        void* at = bytes_of(pages, "pages");
        const uint32_t window = g[8] ? whole(g[8], "window") : 0, sinks = g[9] ? whole(g[9], "sinks") : 0;
        const Attend x(a, spec.head_dim, g[2], g[6], g[7], g[10], g[11], g[12]);
        const at::Tensor& starts = a.need(g[3], "starts");
        if (starts.dim() != 1 || starts.size(0) < 1) refuse("starts: expected int32 [sequences + 1]");
        const int64_t n = starts.size(0) - 1;
        const auto* st = static_cast<const int32_t*>(plain(starts, at::kInt, {n + 1}, "starts"));
        const Table t(a, g[4], g[5], n);
        const uint32_t seqs = count32(n, "starts");
        const size_t size = (size_t)pages.numel();
        return launch("kvpage_attend_prompt", a, g[13], [&](hipStream_t s) {
            return f_page_attend_prompt(&spec, at, size, seqs, x.n, x.hq, &x.q, st, t.table, t.cols, t.stride, t.lens, window,
                                        sinks, x.scale, &x.out, x.lse, x.ws, x.ws_bytes, x.status, s);
        });
    });
}

const char kPoolDoc[] =
    "kvpool_attend(shape, pool, layer, q, out, ws, tail=None, lse=None, scale=None, dev_status=None, stream=None)\n\n"
    "q, out: rows [n_agents, q_heads, head_dim]; pool: uint8 tensor as kvpool_encode wrote it; tail: (spec, pages,\n"
    "table, lens) of the agents' own pages or None; the rest as for kvpage_attend.";
PyObject* pool_attend(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
    return guarded([&]() -> PyObject* {
        static const char* const names[11] = {"shape", "pool", "layer", "q", "out", "ws", "tail", "lse", "scale", "dev_status",
                                              "stream"};
        Args<11> a("kvpool_attend", names, 11, 6, args, nargs, kwnames);
        PyObject** g = a.given;
        if (!g[0] || !g[2]) refuse("shape and layer are required");
        const kvc_shape shape = shape_of(g[0]);
        const uint32_t layer = whole(g[2], "layer");
        const at::Tensor& pool = a.need(g[1], "pool");
        void* at = bytes_of(pool, "pool");
        const Attend x(a, shape.head_dim, g[3], g[4], g[5], g[7], g[8], g[9]);
        kvc_pages spec;
        kvc_tail tail;
        if (g[6]) {
            if (!PyTuple_Check(g[6]) || PyTuple_GET_SIZE(g[6]) != 4) refuse("tail: expected (spec, pages, table, lens)");
            spec = spec_of(PyTuple_GET_ITEM(g[6], 0));
            const at::Tensor& pages = a.need(PyTuple_GET_ITEM(g[6], 1), "tail pages");
            const Table t(a, PyTuple_GET_ITEM(g[6], 2), PyTuple_GET_ITEM(g[6], 3), x.n);
            tail = kvc_tail{&spec, bytes_of(pages, "tail pages"), (size_t)pages.numel(), t.table, t.cols, t.stride, t.lens};
        }
        const size_t size = (size_t)pool.numel();
        return launch("kvpool_attend", a, g[10], [&](hipStream_t s) {
            return f_pool_attend(&shape, at, size, layer, x.n, x.hq, &x.q, x.scale, g[6] ? &tail : nullptr, &x.out, x.lse, x.ws,
                                 x.ws_bytes, x.status, s);
        });
    });
}

template <class F>
bool take_address(F& f, PyObject* o) {
    const size_t v = PyLong_AsSize_t(o);
    if (PyErr_Occurred()) return false;
    f = reinterpret_cast<F>(v);
    return true;
}

// setup(KvcError, raw_stream, device, device_guard, as_floats, the entry points' addresses...)
PyObject* setup(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    PyObject** to[5] = {&g_kvc_error, &g_raw_stream, &g_device, &g_device_guard, &g_as_floats};
    if (nargs != 13) {
        PyErr_SetString(PyExc_TypeError, "setup takes 13 arguments");
        return nullptr;
    }
    if (!take_address(f_norm_rotate, args[5]) || !take_address(f_page_write, args[6]) || !take_address(f_page_read, args[7]) ||
        !take_address(f_page_attend, args[8]) || !take_address(f_pool_attend, args[9]) || !take_address(f_page_append, args[10]) ||
        !take_address(f_page_attend_window, args[11]) || !take_address(f_page_attend_prompt, args[12]))
        return nullptr;
    for (int i = 0; i < 5; ++i) {
        Py_INCREF(args[i]);
        Py_XSETREF(*to[i], args[i]);
    }
    Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL | METH_KEYWORDS
PyMethodDef methods[] = {
    {"kvc_norm_rotate", FAST(norm_rotate), kRotateDoc},
    {"kvpage_write", FAST(page_copy<true>), kWriteDoc},
    {"kvpage_read", FAST(page_copy<false>), kReadDoc},
    {"kvpage_attend", FAST(page_attend), kPageDoc},
    {"kvpool_attend", FAST(pool_attend), kPoolDoc},
    {"kvpage_append", FAST(page_append), kAppendDoc},
    {"kvpage_attend_window", FAST(page_attend_window), kWindowDoc},
    {"kvpage_attend_prompt", FAST(page_attend_prompt), kPromptDoc},
    {"setup", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(setup)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kvattend", "Calls of include/kvattend.h on torch tensors.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__kvattend(void) { return PyModule_Create(&module); }
