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

#include "../../include/qmv.h"

namespace {

decltype(&attn_rope_append) g_rope;
decltype(&attn_tree) g_tree;
decltype(&attn_tree_workspace_bytes) g_tree_ws;
decltype(&attn_evict) g_evict;
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
    if (device >= 0 && x.get_device() != device) value_error(name, "on the cache's device");
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

// (cache, device, q, k, v, pos, inv_freq, table, ctx, cu, interleaved, mscale,
//  q_out, acc, status, stream)
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<16>(n, [&]() -> PyObject * {
        const qmv_attn_cache *c = as_cache(a[0]);
        const Device dev(as_int(a[1]));
        const at::ScalarType kind = kind_of(c);
        if (!THPVariable_Check(a[2])) type_error("q", "a tensor");
        const at::ScalarType in = THPVariable_Unpack(a[2]).scalar_type();
        if (in != at::kFloat && in != kind) type_error("q", "float32 or of the cache's type");
        const at::Tensor &q = tensor(a[2], in, dev, "q"), &k = tensor(a[3], in, dev, "k"),
                         &v = tensor(a[4], in, dev, "v");
        if (q.dim() != 3) value_error("q", "[N][Hq][D]");
        const int64_t N = q.size(0), Hq = q.size(1);
        if (N > INT32_MAX || Hq > INT32_MAX) value_error("q", "smaller");
        const int64_t qs = token_stride(q, N, Hq, c->D, "q"),
                      ks = token_stride(k, N, c->Hkv, c->D, "k"),
                      vs = token_stride(v, N, c->Hkv, c->D, "v");
        const auto *pos = static_cast<const int32_t *>(addr(a[5], at::kInt, N, dev, "pos"));
        const auto *f = static_cast<const double *>(addr(a[6], at::kDouble, -1, dev, "inv_freq"));
        const int64_t half = THPVariable_Unpack(a[6]).numel();
        const Table t = table(a[7], dev, "table");
        const auto *ctx = static_cast<const int32_t *>(addr(a[8], at::kInt, t.B, dev, "ctx"));
        const auto *cu = static_cast<const int32_t *>(addr(a[9], at::kInt, t.B + 1, dev, "cu"));
        const int inter = PyObject_IsTrue(a[10]);
        if (inter < 0) throw Bad();
        const float mscale = (float)as_double(a[11]);
        void *acc = opt(a[13], at::kFloat, slots(c), dev, "acc");
        void *status = opt(a[14], at::kInt, 1, dev, "status");
        at::Tensor made;
        void *out;
        if (a[12] == Py_None) {
            made = make({N, Hq, c->D}, kind, dev);
            out = made.data_ptr();
        } else {
            out = addr(a[12], kind, N * Hq * c->D, dev, "q_out");
        }
        check("attn_rope_append",
              g_rope(c, q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                     in == at::kFloat ? QMV_F32 : c->dtype, (int)Hq, pos, f,
                     half > 65536 ? 1 << 17 : (int)(2 * half), inter, mscale, t.p, t.width, ctx, cu,
                     t.B, (int)N, out, static_cast<float *>(acc), static_cast<int32_t *>(status),
                     as_stream(a[15], dev)));
        return wrap(a[12], made);
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

// (QmvError, address of each entry point)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded<5>(n, [&]() -> PyObject * {
        Py_XDECREF(g_error);
        Py_INCREF(a[0]);
        g_error = a[0];
        g_rope = reinterpret_cast<decltype(g_rope)>(PyLong_AsVoidPtr(a[1]));
        g_tree = reinterpret_cast<decltype(g_tree)>(PyLong_AsVoidPtr(a[2]));
        g_tree_ws = reinterpret_cast<decltype(g_tree_ws)>(PyLong_AsVoidPtr(a[3]));
        g_evict = reinterpret_cast<decltype(g_evict)>(PyLong_AsVoidPtr(a[4]));
        if (PyErr_Occurred()) throw Bad();
        Py_RETURN_NONE;
    });
}

PyCFunction fast(PyObject *(*f)(PyObject *, PyObject *const *, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f));
}

PyMethodDef methods[] = {{"init", fast(init), METH_FASTCALL, nullptr},
                         {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
                         {"tree", fast(tree), METH_FASTCALL, nullptr},
                         {"evict", fast(evict), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_qmv_torch", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__qmv_torch() { return PyModule_Create(&module); }
