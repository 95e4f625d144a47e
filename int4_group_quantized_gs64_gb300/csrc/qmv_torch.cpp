// qmv_torch.cpp - the attention entry points for torch tensors (a CPython
// module). A one-token call takes a few microseconds on the GPU; checking its
// tensors attribute by attribute from Python takes ten more on the host, so
// the checks and the marshalling are here. The computation is behind the C ABI
// of include/qmv.h, whose entry points init() gets as addresses.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <type_traits>

#include "../../include/qmv.h"

namespace {

decltype(&attn_rope_append) g_rope;
decltype(&attn_norm_rope_append) g_norm_rope;
decltype(&attn_tree) g_tree;
decltype(&attn_tree_workspace_bytes) g_tree_ws;
decltype(&attn_window) g_window;
decltype(&attn_window_workspace_bytes) g_window_ws;
decltype(&attn_evict) g_evict;
decltype(&attn_pages_update) g_update;
decltype(&attn_pages_update_workspace_bytes) g_update_ws;
decltype(&attn_pages_fork) g_fork;
decltype(&attn_pages_fork_workspace_bytes) g_fork_ws;
decltype(&attn_pages_copy) g_copy;
decltype(&attn_compact) g_compact;
PyObject *g_error;  // QmvError(name, status)

struct Bad : std::exception {};  // a Python error is set

[[noreturn]] void type_error(const char *name, const char *want) {
    PyErr_Format(PyExc_TypeError, "%s must be %s", name, want);
    throw Bad();
}
[[noreturn]] void value_error(const char *name, const char *want) {
    PyErr_Format(PyExc_ValueError, "%s must be %s", name, want);
    throw Bad();
}

const char *name_of(at::ScalarType t) {
    switch (t) {
        case at::kInt: return "an int32 CUDA tensor";
        case at::kFloat: return "a float32 CUDA tensor";
        case at::kDouble: return "a float64 CUDA tensor";
        case at::kByte: return "a uint8 CUDA tensor";
        case at::kBFloat16: return "a bfloat16 CUDA tensor";
        default: return "a float16 CUDA tensor";
    }
}

const at::Tensor &tensor(PyObject *o, at::ScalarType t, int device, const char *name) {
    if (!THPVariable_Check(o)) type_error(name, name_of(t));
    const at::Tensor &x = THPVariable_Unpack(o);
    if (!x.is_cuda() || x.scalar_type() != t) type_error(name, name_of(t));
    if (device >= 0 && x.get_device() != device) value_error(name, "on the device of the call's cache or pages");
    return x;
}

// The address of a contiguous tensor of n elements (n < 0: any number).
void *addr(PyObject *o, at::ScalarType t, int64_t n, int device, const char *name) {
    const at::Tensor &x = tensor(o, t, device, name);
    if (!x.is_contiguous()) value_error(name, "contiguous");
    if (n >= 0 && x.numel() != n) {
        PyErr_Format(PyExc_ValueError, "%s must have %lld elements, got %lld", name, (long long)n,
                     (long long)x.numel());
        throw Bad();
    }
    return x.data_ptr();
}
void *opt(PyObject *o, at::ScalarType t, int64_t n, int device, const char *name) {
    return o == Py_None ? nullptr : addr(o, t, n, device, name);
}

// [n][heads][D] with a token's heads contiguous: the elements between tokens.
int64_t token_stride(const at::Tensor &x, int64_t n, int64_t heads, int64_t D, const char *name) {
    if (x.dim() != 3 || x.size(0) != n || x.size(1) != heads || x.size(2) != D) {
        PyErr_Format(PyExc_ValueError, "%s must be [%lld][%lld][%lld]", name, (long long)n,
                     (long long)heads, (long long)D);
        throw Bad();
    }
    if (x.stride(2) != 1 || (heads > 1 && x.stride(1) != D))
        value_error(name, "contiguous within a token");
    return n > 1 ? x.stride(0) : heads * D;
}

struct Table {
    const int32_t *p;
    int B, width;
};
Table table(PyObject *o, int device, const char *name) {
    const at::Tensor &x = tensor(o, at::kInt, device, name);
    if (x.dim() != 2 || !x.is_contiguous()) value_error(name, "[B][max_pages] and contiguous");
    if (x.size(0) > INT32_MAX || x.size(1) > INT32_MAX) value_error(name, "smaller");
    return Table{x.data_ptr<int32_t>(), (int)x.size(0), (int)x.size(1)};
}

// The device of a call's cache, which the calls below launch on and ask for
// its number of SMs: current from here to the end of the call.
struct Device {
    int index;
    c10::cuda::CUDAGuard guard;
    explicit Device(int i) : index(i), guard((c10::DeviceIndex)i) {}
    operator int() const { return index; }
};

int as_int(PyObject *o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Bad();
    if (v < INT32_MIN || v > INT32_MAX) {
        PyErr_SetString(PyExc_OverflowError, "a count does not fit 32 bits");
        throw Bad();
    }
    return (int)v;
}
double as_double(PyObject *o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Bad();
    return v;
}
const qmv_attn_cache *as_cache(PyObject *o) {
    void *p = PyLong_AsVoidPtr(o);
    if (!p) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "no cache");
        throw Bad();
    }
    return static_cast<const qmv_attn_cache *>(p);
}
// A stream handle, or None: the current stream of the device.
qmv_stream_t as_stream(PyObject *o, int device) {
    if (o == Py_None)
        return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
    void *p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred()) throw Bad();
    return static_cast<qmv_stream_t>(p);
}
void check(const char *fn, int status) {
    if (status == 0) return;
    PyObject *e = PyObject_CallFunction(g_error, "si", fn, status);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Bad();
}
at::ScalarType kind_of(const qmv_attn_cache *c) {
    return c->dtype == QMV_BF16 ? at::kBFloat16 : at::kHalf;
}
int64_t slots(const qmv_attn_cache *c) { return (int64_t)c->pages * c->Hkv * c->page; }

at::Tensor make(at::IntArrayRef shape, at::ScalarType t, int device) {
    return at::empty(shape, at::TensorOptions().dtype(t).device(at::kCUDA, (c10::DeviceIndex)device));
}

template <int kArgs, class F>
PyObject *guarded(Py_ssize_t n, F &&f) {
    if (n != kArgs) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", kArgs, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Bad &) {
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    }
    return nullptr;
}

PyObject *wrap(PyObject *given, const at::Tensor &made) {
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
}
PyObject *pair(PyObject *a, PyObject *b) {
    PyObject *r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
    Py_XDECREF(a);
    Py_XDECREF(b);
    return r;
}

// The tensors that both rotary appends take, checked: a[at] .. a[at + 10] are
// pos, inv_freq, table, ctx, cu, interleaved, mscale, q_out, acc, status, stream.
struct Append {
    const qmv_attn_cache *c;
    Device dev;
    at::ScalarType kind;
    int64_t N, Hq;
    const void *q, *k, *v;
    int64_t qs, ks, vs;
    int in_dtype, rot, inter;
    const int32_t *pos, *ctx, *cu;
    const double *f;
    Table t;
    float mscale;
    at::Tensor made;
    void *out;
    float *acc;
    int32_t *status;
    qmv_stream_t stream;

    Append(PyObject *const *a, int at)
        : c(as_cache(a[0])), dev(as_int(a[1])), kind(kind_of(c)) {
        if (!THPVariable_Check(a[2])) type_error("q", "a tensor");
        const at::ScalarType in = THPVariable_Unpack(a[2]).scalar_type();
        if (in != at::kFloat && in != kind) type_error("q", "float32 or of the cache's type");
        const at::Tensor &qt = tensor(a[2], in, dev, "q"), &kt = tensor(a[3], in, dev, "k"),
                         &vt = tensor(a[4], in, dev, "v");
        if (qt.dim() != 3) value_error("q", "[N][Hq][D]");
        N = qt.size(0);
        Hq = qt.size(1);
        if (N > INT32_MAX || Hq > INT32_MAX) value_error("q", "smaller");
        qs = token_stride(qt, N, Hq, c->D, "q");
        ks = token_stride(kt, N, c->Hkv, c->D, "k");
        vs = token_stride(vt, N, c->Hkv, c->D, "v");
        q = qt.data_ptr();
        k = kt.data_ptr();
        v = vt.data_ptr();
        in_dtype = in == at::kFloat ? QMV_F32 : c->dtype;
        a += at;
        pos = static_cast<const int32_t *>(addr(a[0], at::kInt, N, dev, "pos"));
        f = static_cast<const double *>(addr(a[1], at::kDouble, -1, dev, "inv_freq"));
        const int64_t half = THPVariable_Unpack(a[1]).numel();
        rot = half > 65536 ? 1 << 17 : (int)(2 * half);
        t = table(a[2], dev, "table");
        ctx = static_cast<const int32_t *>(addr(a[3], at::kInt, t.B, dev, "ctx"));
        cu = static_cast<const int32_t *>(addr(a[4], at::kInt, t.B + 1, dev, "cu"));
        inter = PyObject_IsTrue(a[5]);
        if (inter < 0) throw Bad();
        mscale = (float)as_double(a[6]);
        acc = static_cast<float *>(opt(a[8], at::kFloat, slots(c), dev, "acc"));
        status = static_cast<int32_t *>(opt(a[9], at::kInt, 1, dev, "status"));
        if (a[7] == Py_None) {
            made = make({N, Hq, c->D}, kind, dev);
            out = made.data_ptr();
        } else {
            out = addr(a[7], kind, N * Hq * c->D, dev, "q_out");
        }
        stream = as_stream(a[10], dev);
    }
};

// (cache, device, q, k, v, pos, inv_freq, table, ctx, cu, interleaved, mscale,
//  q_out, acc, status, stream)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<16>(n, [&]() -> PyObject * {
        const Append x(a, 5);
        check("attn_rope_append",
              g_rope(x.c, x.q, x.qs, x.k, x.ks, x.v, x.vs, x.in_dtype, (int)x.Hq, x.pos, x.f, x.rot,
                     x.inter, x.mscale, x.t.p, x.t.width, x.ctx, x.cu, x.t.B, (int)x.N, x.out, x.acc,
                     x.status, x.stream));
        return wrap(a[12], x.made);
    });
}

// (cache, device, q, k, v, q_weight, k_weight, eps, pos, inv_freq, table, ctx, cu,
//  interleaved, mscale, q_out, acc, status, stream)
PyObject *norm_rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<19>(n, [&]() -> PyObject * {
        const Append x(a, 8);
        // both weights in one type (that of the first that is there)
        at::ScalarType wk = at::kFloat;
        for (int i = 6; i >= 5; --i)
            if (a[i] != Py_None) {
                if (!THPVariable_Check(a[i])) type_error(i == 5 ? "q_weight" : "k_weight", "a tensor");
                wk = THPVariable_Unpack(a[i]).scalar_type();
            }
        if (wk != at::kFloat && wk != x.kind) type_error("q_weight and k_weight", "float32 or of the cache's type");
        const void *qw = opt(a[5], wk, x.c->D, x.dev, "q_weight"), *kw = opt(a[6], wk, x.c->D, x.dev, "k_weight");
        check("attn_norm_rope_append",
              g_norm_rope(x.c, x.q, x.qs, x.k, x.ks, x.v, x.vs, x.in_dtype, (int)x.Hq, qw, kw,
                          wk == at::kFloat ? QMV_F32 : x.c->dtype, (float)as_double(a[7]), x.pos, x.f,
                          x.rot, x.inter, x.mscale, x.t.p, x.t.width, x.ctx, x.cu, x.t.B, (int)x.N,
                          x.out, x.acc, x.status, x.stream));
        return wrap(a[15], x.made);
    });
}

// (cache, device, q, table, ctx, cu, max_draft, mask, scale, o, o_float32, lse,
//  acc, acc_out, decay, ws, status, stream)
PyObject *tree(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<18>(n, [&]() -> PyObject * {
        const qmv_attn_cache *c = as_cache(a[0]);
        const Device dev(as_int(a[1]));
        const at::ScalarType kind = kind_of(c);
        const at::Tensor &q = tensor(a[2], kind, dev, "q");
        if (q.dim() != 3) value_error("q", "[N][Hq][D]");
        const int64_t N = q.size(0), Hq = q.size(1);
        if (N > INT32_MAX || Hq > INT32_MAX) value_error("q", "smaller");
        const int64_t qs = token_stride(q, N, Hq, c->D, "q");
        const Table t = table(a[3], dev, "table");
        const auto *ctx = static_cast<const int32_t *>(addr(a[4], at::kInt, t.B, dev, "ctx"));
        const auto *cu = static_cast<const int32_t *>(addr(a[5], at::kInt, t.B + 1, dev, "cu"));
        const int max_draft = as_int(a[6]);
        const uint32_t *mask = nullptr;
        int words = 0;
        if (a[7] != Py_None) {
            const at::Tensor &m = tensor(a[7], at::kInt, dev, "mask");
            if (m.dim() != 2 || m.size(0) != N || !m.is_contiguous() || m.size(1) > 1 << 20)
                value_error("mask", "[N][words] and contiguous");
            mask = reinterpret_cast<const uint32_t *>(m.data_ptr<int32_t>());
            words = (int)m.size(1);
        }
        const float scale = (float)as_double(a[8]), decay = (float)as_double(a[14]);
        const int f32 = PyObject_IsTrue(a[10]);
        if (f32 < 0) throw Bad();
        const at::ScalarType okind = f32 ? at::kFloat : kind;
        auto *acc = static_cast<float *>(opt(a[12], at::kFloat, slots(c), dev, "acc"));
        auto *acc_out = static_cast<float *>(opt(a[13], at::kFloat, slots(c), dev, "acc_out"));
        void *status = opt(a[16], at::kInt, 1, dev, "status");
        at::Tensor made_o, made_lse, made_ws;
        void *o, *lse, *ws;
        size_t ws_bytes;
        if (a[9] == Py_None) {
            made_o = make({N, Hq, c->D}, okind, dev);
            o = made_o.data_ptr();
        } else {
            o = addr(a[9], okind, N * Hq * c->D, dev, "o");
        }
        if (a[11] == Py_None) {
            made_lse = make({N, Hq}, at::kFloat, dev);
            lse = made_lse.data_ptr();
        } else {
            lse = addr(a[11], at::kFloat, N * Hq, dev, "lse");
        }
        if (a[15] == Py_None) {
            ws_bytes = g_tree_ws(c, (int)Hq, t.B, (int)N, max_draft, t.width, acc_out != nullptr);
            made_ws = make({(int64_t)(ws_bytes < 256 ? 256 : ws_bytes)}, at::kByte, dev);
            ws = made_ws.data_ptr();
        } else {
            ws = addr(a[15], at::kByte, -1, dev, "ws");
            ws_bytes = (size_t)THPVariable_Unpack(a[15]).numel();
        }
        check("attn_tree",
              g_tree(c, q.data_ptr(), qs, (int)Hq, t.p, t.width, ctx, cu, t.B, (int)N, max_draft, mask,
                     words, scale, o, f32 ? QMV_F32 : c->dtype, static_cast<float *>(lse), acc, acc_out,
                     decay, static_cast<int32_t *>(status), ws, ws_bytes, as_stream(a[17], dev)));
        return pair(wrap(a[9], made_o), wrap(a[11], made_lse));
    });
}

// (cache, device, q, table, ctx, cu, max_new, window, sinks, scale, o, o_float32,
//  lse, ws, status, stream)
PyObject *window(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<16>(n, [&]() -> PyObject * {
        const qmv_attn_cache *c = as_cache(a[0]);
        const Device dev(as_int(a[1]));
        const at::ScalarType kind = kind_of(c);
        const at::Tensor &q = tensor(a[2], kind, dev, "q");
        if (q.dim() != 3) value_error("q", "[N][Hq][D]");
        const int64_t N = q.size(0), Hq = q.size(1);
        if (N > INT32_MAX || Hq > INT32_MAX) value_error("q", "smaller");
        const int64_t qs = token_stride(q, N, Hq, c->D, "q");
        const Table t = table(a[3], dev, "table");
        const auto *ctx = static_cast<const int32_t *>(addr(a[4], at::kInt, t.B, dev, "ctx"));
        const auto *cu = static_cast<const int32_t *>(addr(a[5], at::kInt, t.B + 1, dev, "cu"));
        const int max_new = as_int(a[6]), win = as_int(a[7]), sinks = as_int(a[8]);
        const float scale = (float)as_double(a[9]);
        const int f32 = PyObject_IsTrue(a[11]);
        if (f32 < 0) throw Bad();
        const at::ScalarType okind = f32 ? at::kFloat : kind;
        void *status = opt(a[14], at::kInt, 1, dev, "status");
        at::Tensor made_o, made_lse, made_ws;
        void *o, *lse, *ws;
        size_t ws_bytes;
        if (a[10] == Py_None) {
            made_o = make({N, Hq, c->D}, okind, dev);
            o = made_o.data_ptr();
        } else {
            o = addr(a[10], okind, N * Hq * c->D, dev, "o");
        }
        if (a[12] == Py_None) {
            made_lse = make({N, Hq}, at::kFloat, dev);
            lse = made_lse.data_ptr();
        } else {
            lse = addr(a[12], at::kFloat, N * Hq, dev, "lse");
        }
        if (a[13] == Py_None) {
            ws_bytes = g_window_ws(c, (int)Hq, t.B, (int)N, max_new, t.width);
            made_ws = make({(int64_t)(ws_bytes < 256 ? 256 : ws_bytes)}, at::kByte, dev);
            ws = made_ws.data_ptr();
        } else {
            ws = addr(a[13], at::kByte, -1, dev, "ws");
            ws_bytes = (size_t)THPVariable_Unpack(a[13]).numel();
        }
        check("attn_window",
              g_window(c, q.data_ptr(), qs, (int)Hq, t.p, t.width, ctx, cu, t.B, (int)N, max_new, win,
                       sinks, scale, o, f32 ? QMV_F32 : c->dtype, static_cast<float *>(lse),
                       static_cast<int32_t *>(status), ws, ws_bytes, as_stream(a[15], dev)));
        return pair(wrap(a[10], made_o), wrap(a[12], made_lse));
    });
}

// (src, device, acc, table, lens, budget, dst, dst_acc, dst_table, sink, recent,
//  keep, new_lens, status, stream)
PyObject *evict(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<15>(n, [&]() -> PyObject * {
        const qmv_attn_cache *c = as_cache(a[0]), *d = as_cache(a[6]);
        const Device dev(as_int(a[1]));
        const auto *acc = static_cast<const float *>(addr(a[2], at::kFloat, slots(c), dev, "acc"));
        const Table t = table(a[3], dev, "table");
        const auto *lens = static_cast<const int32_t *>(addr(a[4], at::kInt, t.B, dev, "lens"));
        const int budget = as_int(a[5]);
        auto *dacc = static_cast<float *>(addr(a[7], at::kFloat, slots(d), dev, "dst_acc"));
        const Table dt = table(a[8], dev, "dst_table");
        if (dt.B != t.B) value_error("dst_table", "as many rows as table");
        const int sink = as_int(a[9]), recent = as_int(a[10]);
        const int64_t kept = budget > 0 ? budget : 0;
        void *status = opt(a[13], at::kInt, 1, dev, "status");
        at::Tensor made_keep, made_lens;
        void *keep, *new_lens;
        if (a[11] == Py_None) {
            made_keep = make({t.B, c->Hkv, kept}, at::kInt, dev);
            keep = made_keep.data_ptr();
        } else {
            keep = addr(a[11], at::kInt, t.B * c->Hkv * kept, dev, "keep");
        }
        if (a[12] == Py_None) {
            made_lens = make({t.B}, at::kInt, dev);
            new_lens = made_lens.data_ptr();
        } else {
            new_lens = addr(a[12], at::kInt, t.B, dev, "new_lens");
        }
        check("attn_evict",
              g_evict(c, acc, t.p, t.width, lens, t.B, budget, sink, recent, d, dacc, dt.p, dt.width,
                      static_cast<int32_t *>(keep), static_cast<int32_t *>(new_lens),
                      static_cast<int32_t *>(status), as_stream(a[14], dev)));
        return pair(wrap(a[11], made_keep), wrap(a[12], made_lens));
    });
}

// The counts of a pool's pages: their number, and the device that they are on.
struct Refs {
    int32_t *p;
    int pages, device;
};
Refs refs(PyObject *o) {
    const at::Tensor &x = tensor(o, at::kInt, -1, "refs");
    if (x.dim() != 1 || !x.is_contiguous()) value_error("refs", "[pages] and contiguous");
    if (x.size(0) > INT32_MAX) value_error("refs", "smaller");
    return Refs{x.data_ptr<int32_t>(), (int)x.size(0), (int)x.get_device()};
}
// A given workspace, or one made for the call.
struct Workspace {
    at::Tensor made;
    void *p;
    size_t bytes;
    Workspace(PyObject *o, size_t want, int device) {
        if (o == Py_None) {
            bytes = want < 256 ? 256 : want;
            made = make({(int64_t)bytes}, at::kByte, device);
            p = made.data_ptr();
        } else {
            p = addr(o, at::kByte, -1, device, "ws");
            bytes = (size_t)THPVariable_Unpack(o).numel();
        }
    }
};
// A given int32 output of this many elements, or one made with this shape.
struct Out {
    at::Tensor made;
    int32_t *p;
    Out(PyObject *o, at::IntArrayRef shape, int device, const char *name) {
        int64_t n = 1;
        for (const int64_t d : shape) n *= d;
        if (o == Py_None) {
            made = make(shape, at::kInt, device);
            p = made.data_ptr<int32_t>();
        } else {
            p = static_cast<int32_t *>(addr(o, at::kInt, n, device, name));
        }
    }
};

// (refs, table, lens, more, page, window, sinks, ws, status, stream)
PyObject *pages_update(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<10>(n, [&]() -> PyObject * {
        const Refs r = refs(a[0]);
        const Device dev(r.device);
        const Table t = table(a[1], dev, "table");
        const auto *lens = static_cast<const int32_t *>(addr(a[2], at::kInt, t.B, dev, "lens"));
        const auto *more = static_cast<const int32_t *>(addr(a[3], at::kInt, t.B, dev, "more"));
        const int page = as_int(a[4]), win = as_int(a[5]), sinks = as_int(a[6]);
        const Workspace ws(a[7], g_update_ws(r.pages, t.B, t.width), dev);
        void *status = opt(a[8], at::kInt, 1, dev, "status");
        check("attn_pages_update",
              g_update(r.p, r.pages, page, const_cast<int32_t *>(t.p), t.width, lens, more, t.B, win,
                       sinks, static_cast<int32_t *>(status), ws.p, ws.bytes, as_stream(a[9], dev)));
        Py_RETURN_NONE;
    });
}

// (refs, table, lens, parent, page, new_table, new_lens, moves, ws, status, stream)
PyObject *pages_fork(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<11>(n, [&]() -> PyObject * {
        const Refs r = refs(a[0]);
        const Device dev(r.device);
        const Table t = table(a[1], dev, "table");
        const auto *lens = static_cast<const int32_t *>(addr(a[2], at::kInt, t.B, dev, "lens"));
        const auto *parent = static_cast<const int32_t *>(addr(a[3], at::kInt, -1, dev, "parent"));
        const int64_t F = THPVariable_Unpack(a[3]).numel();
        if (F > INT32_MAX) value_error("parent", "smaller");
        const int page = as_int(a[4]);
        const Out table2(a[5], {F, t.width}, dev, "new_table"), lens2(a[6], {F}, dev, "new_lens"),
            moves(a[7], {F, 3}, dev, "moves");
        const Workspace ws(a[8], g_fork_ws(r.pages, (int)F), dev);
        void *status = opt(a[9], at::kInt, 1, dev, "status");
        check("attn_pages_fork",
              g_fork(r.p, r.pages, page, t.p, t.width, lens, t.B, parent, (int)F, table2.p, lens2.p,
                     moves.p, static_cast<int32_t *>(status), ws.p, ws.bytes, as_stream(a[10], dev)));
        PyObject *x = wrap(a[5], table2.made), *y = wrap(a[6], lens2.made), *z = wrap(a[7], moves.made);
        PyObject *res = x && y && z ? PyTuple_Pack(3, x, y, z) : nullptr;
        Py_XDECREF(x);
        Py_XDECREF(y);
        Py_XDECREF(z);
        return res;
    });
}

// (src, dst, device, moves, src_acc, dst_acc, status, stream)
PyObject *pages_copy(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<8>(n, [&]() -> PyObject * {
        const qmv_attn_cache *s = as_cache(a[0]), *d = as_cache(a[1]);
        const Device dev(as_int(a[2]));
        const at::Tensor &m = tensor(a[3], at::kInt, dev, "moves");
        if (m.dim() != 2 || m.size(1) != 3 || !m.is_contiguous()) value_error("moves", "[n][3] and contiguous");
        if (m.size(0) > INT32_MAX) value_error("moves", "smaller");
        const auto *sacc = static_cast<const float *>(opt(a[4], at::kFloat, slots(s), dev, "src_acc"));
        auto *dacc = static_cast<float *>(opt(a[5], at::kFloat, slots(d), dev, "dst_acc"));
        void *status = opt(a[6], at::kInt, 1, dev, "status");
        check("attn_pages_copy", g_copy(s, d, m.data_ptr<int32_t>(), (int)m.size(0), sacc, dacc,
                                        static_cast<int32_t *>(status), as_stream(a[7], dev)));
        Py_RETURN_NONE;
    });
}

// (cache, device, table, ctx, cu, keep, kept, acc, new_ctx, status, stream)
PyObject *compact(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<11>(n, [&]() -> PyObject * {
        const qmv_attn_cache *c = as_cache(a[0]);
        const Device dev(as_int(a[1]));
        const Table t = table(a[2], dev, "table");
        const auto *ctx = static_cast<const int32_t *>(addr(a[3], at::kInt, t.B, dev, "ctx"));
        const auto *cu = static_cast<const int32_t *>(addr(a[4], at::kInt, t.B + 1, dev, "cu"));
        const auto *keep = static_cast<const int32_t *>(addr(a[5], at::kInt, -1, dev, "keep"));
        const int64_t N = THPVariable_Unpack(a[5]).numel();
        if (N > INT32_MAX) value_error("keep", "smaller");
        const auto *kept = static_cast<const int32_t *>(addr(a[6], at::kInt, t.B, dev, "kept"));
        auto *acc = static_cast<float *>(opt(a[7], at::kFloat, slots(c), dev, "acc"));
        const Out now(a[8], {t.B}, dev, "new_ctx");
        void *status = opt(a[9], at::kInt, 1, dev, "status");
        check("attn_compact", g_compact(c, t.p, t.width, ctx, cu, t.B, (int)N, keep, kept, acc, now.p,
                                        static_cast<int32_t *>(status), as_stream(a[10], dev)));
        return wrap(a[8], now.made);
    });
}

// (QmvError, address of each entry point)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<14>(n, [&]() -> PyObject * {
        Py_XDECREF(g_error);
        Py_INCREF(a[0]);
        g_error = a[0];
        int i = 1;
        auto take = [&](auto &f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(PyLong_AsVoidPtr(a[i++])); };
        take(g_rope);
        take(g_norm_rope);
        take(g_tree);
        take(g_tree_ws);
        take(g_window);
        take(g_window_ws);
        take(g_evict);
        take(g_update);
        take(g_update_ws);
        take(g_fork);
        take(g_fork_ws);
        take(g_copy);
        take(g_compact);
        if (PyErr_Occurred()) throw Bad();
        Py_RETURN_NONE;
    });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"init", fast(init), METH_FASTCALL, nullptr},
                         {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
                         {"norm_rope_append", fast(norm_rope_append), METH_FASTCALL, nullptr},
                         {"tree", fast(tree), METH_FASTCALL, nullptr},
                         {"window", fast(window), METH_FASTCALL, nullptr},
                         {"evict", fast(evict), METH_FASTCALL, nullptr},
                         {"pages_update", fast(pages_update), METH_FASTCALL, nullptr},
                         {"pages_fork", fast(pages_fork), METH_FASTCALL, nullptr},
                         {"pages_copy", fast(pages_copy), METH_FASTCALL, nullptr},
                         {"compact", fast(compact), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmv_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__qmv_torch() { return PyModule_Create(&module); }
