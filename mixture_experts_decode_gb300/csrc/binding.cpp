// binding.cpp -- CPython module `_block`: argument marshalling of the decode
// block's entry points (moe_paged_attention, moe_rope_append,
// moe_norm_residual, moe_matvec4) and of the serving step's around them
// (moe_shared_prefix_attention, moe_router_grouped_topk, moe_plan_pages,
// moe_release_pages).
//
// These calls are a few microseconds of GPU work for one token, and the same
// checks made in Python through ctypes took 20 to 30 us on the host (a
// Grace core); here they read the tensors' own fields.  Nothing is computed
// here: dtypes, devices, shapes and strides are checked, outputs allocated
// and raw pointers handed to the C ABI with the current stream.
#include <ATen/ATen.h>
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/moedec.h"

namespace {

using at::Tensor;

PyObject* g_fail = nullptr;  // callable (function name, status): raises MoEError

struct Refused {
    PyObject* type;  // borrowed: a builtin exception
    std::string text;
};
struct Raised {};  // a Python exception is set

[[noreturn]] void type_error(const std::string& s) { throw Refused{PyExc_TypeError, s}; }
[[noreturn]] void value_error(const std::string& s) { throw Refused{PyExc_ValueError, s}; }

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}
double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}
int integer(PyObject* o) {
    const long v = PyLong_AsLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX) throw Refused{PyExc_OverflowError, "integer argument beyond 32 bits"};
    return (int)v;
}
bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}
int size32(int64_t n, const char* name) {
    if (n > INT32_MAX) value_error(std::string(name) + " has a dimension beyond 32 bits");
    return (int)n;
}

int dtype_code(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return MOE_BF16;
        case at::kHalf: return MOE_F16;
        case at::kFloat: return MOE_F32;
        case at::kFloat8_e4m3fn: return MOE_E4M3;
        default: return -1;
    }
}
int half_code(const Tensor& t, const char* name) {
    if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
        type_error(std::string(name) + " must be bfloat16 or float16, got " + c10::toString(t.scalar_type()));
    return dtype_code(t.scalar_type());
}
void is(const Tensor& t, const char* name, at::ScalarType type, const at::Device& dev, int64_t ndim) {
    if (t.scalar_type() != type)
        type_error(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (t.device() != dev) value_error(std::string(name) + " must be on " + dev.str() + ", got " + t.device().str());
    if (t.dim() != ndim)
        value_error(std::string(name) + " must have " + std::to_string(ndim) + " dims, got " + std::to_string(t.dim()));
}
void dense(const Tensor& t, const char* name) {
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
}
void last_dense(const Tensor& t, const char* name) {
    const int64_t n = t.dim() - 1;
    if (t.size(n) > 1 && t.stride(n) != 1) value_error(std::string(name) + "'s last dimension must be contiguous");
}
// The stride of a dimension of one element is free: 0 keeps it aligned.
int64_t step_of(const Tensor& t, int64_t dim) { return t.size(dim) > 1 ? t.stride(dim) : 0; }

// [tokens, heads, D] with contiguous heads' rows
void heads(const Tensor& t, const char* name, at::ScalarType type, const at::Device& dev, int64_t n, int64_t h, int64_t d) {
    is(t, name, type, dev, 3);
    if (n >= 0 && (t.size(0) != n || t.size(1) != h || t.size(2) != d))
        value_error(std::string(name) + " must be [" + std::to_string(n) + ", " + std::to_string(h) + ", " +
                    std::to_string(d) + "]");
    last_dense(t, name);
}

struct Caches {
    moe_cache_t k, v;
    int dtype, pages, page, heads;
};
moe_cache_t cache_of(const Tensor& t, double scale) {
    return {t.data_ptr(), step_of(t, 0), step_of(t, 1), step_of(t, 2), (float)scale};
}
Caches caches(const Tensor& k, const Tensor& v, at::ScalarType type, const at::Device& dev, int64_t D, double ks, double vs) {
    const at::ScalarType ct = k.scalar_type();
    if (ct != type && ct != at::kFloat8_e4m3fn)
        type_error(std::string("k_cache must be ") + c10::toString(type) + " or float8_e4m3fn, got " + c10::toString(ct));
    is(k, "k_cache", ct, dev, 4);
    is(v, "v_cache", ct, dev, 4);
    if (k.sizes() != v.sizes() || k.size(3) != D)
        value_error("k_cache and v_cache must be alike, [num_pages, page_size, Hkv, D], and have q's head size");
    last_dense(k, "k_cache");
    last_dense(v, "v_cache");
    return {cache_of(k, ks), cache_of(v, vs), dtype_code(ct), size32(k.size(0), "k_cache"), size32(k.size(1), "k_cache"),
            size32(k.size(2), "k_cache")};
}

// The device's guard and stream; refuses tensors that are not on a GPU.
struct OnDevice {
    c10::cuda::OptionalCUDAGuard guard;
    moe_stream_t stream;
    explicit OnDevice(const at::Device& dev) {
        if (!dev.is_cuda()) value_error("tensors must be on a CUDA device, got " + dev.str());
        guard.set_device(dev);
        stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
};

void check(const char* fn, int rc) {
    if (rc == MOE_OK) return;
    PyObject* r = PyObject_CallFunction(g_fail, "si", fn, rc);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
    throw Raised{};
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
    if (n != want) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
        return nullptr;
    }
    try {
        return f();
    } catch (const Raised&) {
    } catch (const Refused& r) {
        PyErr_SetString(r.type, r.text.c_str());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The caller's output tensor, or a new one.
Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, const at::TensorOptions& opt) {
    if (o == Py_None) return at::empty(shape, opt);
    const Tensor& t = tensor(o, name);
    is(t, name, c10::typeMetaToScalarType(opt.dtype()), opt.device(), (int64_t)shape.size());
    dense(t, name);
    if (t.sizes() != shape) value_error(std::string(name) + " has the wrong shape");
    return t;
}

// q, k_cache, v_cache, block_table, seq_lens, scale, window, sinks, k_scale,
// v_scale, workspace, out, return_lse, lse
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 14, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
        const Tensor &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "seq_lens");
        const int dt = half_code(q, "q");
        const at::ScalarType type = q.scalar_type();
        const at::Device dev = q.device();
        heads(q, "q", type, dev, -1, 0, 0);
        const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
        const Caches c = caches(k, v, type, dev, D, number(a[8]), number(a[9]));
        is(table, "block_table", at::kInt, dev, 2);
        if (table.size(0) != B || (table.size(1) > 1 && table.stride(1) != 1))
            value_error("block_table must be [B, max_pages] with contiguous rows");
        is(lens, "seq_lens", at::kInt, dev, 1);
        dense(lens, "seq_lens");
        if (lens.size(0) != B) value_error("seq_lens must be [B]");
        const double scale = a[5] == Py_None ? 1.0 / std::sqrt((double)D) : number(a[5]);
        const OnDevice on(dev);
        Tensor ws;
        if (a[10] == Py_None) {
            size_t bytes = 0;
            check("moe_paged_attention_workspace_bytes",
                  moe_paged_attention_workspace_bytes(size32(Hq, "q"), c.heads, size32(D, "q"), &bytes));
            ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
            ws.narrow(0, 0, MOE_ATTN_COUNTER_BYTES).zero_();
        } else {
            ws = tensor(a[10], "workspace");
            is(ws, "workspace", at::kByte, dev, 1);
            dense(ws, "workspace");
        }
        const Tensor out = output(a[11], "out", {B, Hq, D}, q.options());
        const bool want = truth(a[12]);
        Tensor lse;
        if (want || a[13] != Py_None) lse = output(a[13], "lse", {B, Hq}, q.options().dtype(at::kFloat));
        check("moe_paged_attention",
              moe_paged_attention(q.data_ptr(), step_of(q, 0), step_of(q, 1), size32(B, "q"), size32(Hq, "q"), c.heads,
                                  size32(D, "q"), dt, c.k, c.v, c.dtype, c.pages, c.page,
                                  static_cast<const int32_t*>(table.data_ptr()), step_of(table, 0),
                                  size32(table.size(1), "block_table"), static_cast<const int32_t*>(lens.data_ptr()),
                                  (float)scale, integer(a[6]), integer(a[7]), ws.data_ptr(), (size_t)ws.numel(),
                                  out.data_ptr(), lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, on.stream));
        if (!want) return THPVariable_Wrap(out);
        PyObject* r = PyTuple_New(2);
        if (!r) throw Raised{};
        PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(out));
        PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(lse));
        return r;
    });
}

// q, k, v, positions, slots, freqs, k_cache, v_cache, interleaved, mscale,
// k_scale, v_scale, q_out
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 13, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
        const Tensor &pos = tensor(a[3], "positions"), &slots = tensor(a[4], "slots"), &freqs = tensor(a[5], "freqs");
        const int dt = half_code(q, "q");
        const at::ScalarType type = q.scalar_type();
        const at::Device dev = q.device();
        heads(q, "q", type, dev, -1, 0, 0);
        const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
        const Caches c = caches(tensor(a[6], "k_cache"), tensor(a[7], "v_cache"), type, dev, D, number(a[10]), number(a[11]));
        heads(k, "k", type, dev, T, c.heads, D);
        heads(v, "v", type, dev, T, c.heads, D);
        is(pos, "positions", at::kInt, dev, 1);
        is(slots, "slots", at::kLong, dev, 1);
        is(freqs, "freqs", at::kDouble, dev, 1);
        dense(pos, "positions");
        dense(slots, "slots");
        dense(freqs, "freqs");
        if (pos.size(0) != T || slots.size(0) != T) value_error("positions and slots must be [T]");
        const OnDevice on(dev);
        Tensor out;
        if (a[12] == Py_None) {
            out = at::empty({T, Hq, D}, q.options());
        } else {
            out = tensor(a[12], "q_out");
            heads(out, "q_out", type, dev, T, Hq, D);
        }
        check("moe_rope_append",
              moe_rope_append(q.data_ptr(), step_of(q, 0), step_of(q, 1), k.data_ptr(), step_of(k, 0), step_of(k, 1),
                              v.data_ptr(), step_of(v, 0), step_of(v, 1), size32(T, "q"), size32(Hq, "q"), c.heads,
                              size32(D, "q"), dt, static_cast<const int32_t*>(pos.data_ptr()),
                              static_cast<const int64_t*>(slots.data_ptr()), static_cast<const double*>(freqs.data_ptr()),
                              2 * size32(freqs.size(0), "freqs"), truth(a[8]) ? 1 : 0, (float)number(a[9]), c.k, c.v, c.dtype,
                              c.pages, c.page, out.data_ptr(), step_of(out, 0), step_of(out, 1), on.stream));
        return THPVariable_Wrap(out);
    });
}

// A Norm tuple (w, b, eps, kind) -> moe_norm_t.
std::optional<moe_norm_t> norm_of(PyObject* o, const char* name, at::ScalarType type, const at::Device& dev, int64_t d) {
    if (o == Py_None) return std::nullopt;
    if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) type_error(std::string(name) + " must be a Norm");
    const void* p[2] = {nullptr, nullptr};
    for (int i = 0; i < 2; ++i) {
        PyObject* part = PyTuple_GET_ITEM(o, i);
        if (part == Py_None) continue;
        const std::string what = std::string(name) + (i ? ".b" : ".w");
        const Tensor& t = tensor(part, what.c_str());
        is(t, what.c_str(), type, dev, 1);
        dense(t, what.c_str());
        if (t.size(0) != d) value_error(what + " must be [" + std::to_string(d) + "]");
        p[i] = t.data_ptr();
    }
    PyObject* kind = PyTuple_GET_ITEM(o, 3);
    int code = -1;
    if (PyUnicode_Check(kind)) {
        if (PyUnicode_CompareWithASCIIString(kind, "rms") == 0) code = MOE_NORM_RMS;
        if (PyUnicode_CompareWithASCIIString(kind, "layer") == 0) code = MOE_NORM_LAYER;
    }
    if (code < 0) {
        PyErr_SetObject(PyExc_KeyError, kind);
        throw Raised{};
    }
    return moe_norm_t{p[0], p[1], (float)number(PyTuple_GET_ITEM(o, 2)), code};
}

// y, resid, post, gate, gate_act, alpha, pre, resid_out, out
PyObject* norm_residual(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 9, [&]() -> PyObject* {
        const Tensor& y = tensor(a[0], "y");
        const int dt = half_code(y, "y");
        const at::ScalarType type = y.scalar_type();
        const at::Device dev = y.device();
        is(y, "y", type, dev, 2);
        last_dense(y, "y");
        const int64_t T = y.size(0), d = y.size(1);
        at::ScalarType rt = type;
        const Tensor* r = nullptr;
        if (a[1] != Py_None) {
            r = &tensor(a[1], "resid");
            rt = r->scalar_type();
            if (rt != type && rt != at::kFloat)
                type_error(std::string("resid must be ") + c10::toString(type) + " or float32, got " + c10::toString(rt));
            is(*r, "resid", rt, dev, 2);
            if (r->sizes() != y.sizes()) value_error("resid must have y's shape");
            last_dense(*r, "resid");
        }
        const auto post = norm_of(a[2], "post", type, dev, d), pre = norm_of(a[6], "pre", type, dev, d);
        const Tensor* g = nullptr;
        int64_t g_row = 0, g_col = 0;
        if (a[3] != Py_None) {
            g = &tensor(a[3], "gate");
            is(*g, "gate", type, dev, 2);
            const int64_t gt = g->size(0), gd = g->size(1);
            if ((gt != 1 && gt != T) || (gd != 1 && gd != d) || (gd > 1 && g->stride(1) != 0 && g->stride(1) != 1))
                value_error("gate must be [T or 1, d or 1] with contiguous rows");
            g_row = step_of(*g, 0);
            g_col = step_of(*g, 1);
        }
        const int act = integer(a[4]);
        const OnDevice on(dev);
        const bool both = r || a[7] != Py_None;
        Tensor ro;
        if (both) ro = output(a[7], "resid_out", {T, d}, y.options().dtype(rt));
        const Tensor out = output(a[8], "out", {T, d}, y.options());
        check("moe_norm_residual",
              moe_norm_residual(y.data_ptr(), step_of(y, 0), size32(T, "y"), size32(d, "y"), dt, r ? r->data_ptr() : nullptr,
                                r ? step_of(*r, 0) : 0, dtype_code(rt), post ? &*post : nullptr,
                                g ? g->data_ptr() : nullptr, g_row, g_col, act, (float)number(a[5]), pre ? &*pre : nullptr,
                                both ? ro.data_ptr() : nullptr, out.data_ptr(), on.stream));
        if (!both) return THPVariable_Wrap(out);
        PyObject* t = PyTuple_New(2);
        if (!t) throw Raised{};
        PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(ro));
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(out));
        return t;
    });
}

// x, W4 tuple (codes, scales, zeros), y
PyObject* matvec4(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 3, [&]() -> PyObject* {
        const Tensor& x = tensor(a[0], "x");
        const int dt = half_code(x, "x");
        const at::ScalarType type = x.scalar_type();
        const at::Device dev = x.device();
        is(x, "x", type, dev, 2);
        last_dense(x, "x");
        const int64_t T = x.size(0), K = x.size(1);
        if (!PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 3) type_error("w must be a W4");
        const Tensor& codes = tensor(PyTuple_GET_ITEM(a[1], 0), "w.codes");
        const Tensor& scales = tensor(PyTuple_GET_ITEM(a[1], 1), "w.scales");
        is(codes, "w.codes", at::kByte, dev, 2);
        is(scales, "w.scales", type, dev, 2);
        dense(codes, "w.codes");
        dense(scales, "w.scales");
        const int64_t N = scales.size(0), groups = scales.size(1);
        if (K % 2 || codes.size(0) != N || codes.size(1) != K / 2 || groups == 0 || K % groups)
            value_error("codes must be [N, K/2] and scales [N, K/group] for x's K = " + std::to_string(K));
        const Tensor* zeros = nullptr;
        if (PyTuple_GET_ITEM(a[1], 2) != Py_None) {
            zeros = &tensor(PyTuple_GET_ITEM(a[1], 2), "w.zeros");
            is(*zeros, "w.zeros", at::kByte, dev, 2);
            dense(*zeros, "w.zeros");
            if (zeros->sizes() != scales.sizes()) value_error("zeros must have the shape of scales");
        }
        const OnDevice on(dev);
        Tensor y;
        if (a[2] == Py_None) {
            y = at::empty({T, N}, x.options());
        } else {
            y = tensor(a[2], "y");
            is(y, "y", type, dev, 2);
            if (y.size(0) != T || y.size(1) != N) value_error("y must be [T, N]");
            last_dense(y, "y");
        }
        check("moe_matvec4",
              moe_matvec4(x.data_ptr(), step_of(x, 0), size32(T, "x"), size32(K, "x"), dt,
                          static_cast<const uint8_t*>(codes.data_ptr()), scales.data_ptr(),
                          zeros ? static_cast<const uint8_t*>(zeros->data_ptr()) : nullptr, size32(N, "scales"),
                          size32(K / groups, "x"), y.data_ptr(), step_of(y, 0), on.stream));
        return THPVariable_Wrap(y);
    });
}

// A uint8 or bool array of B flags.
const uint8_t* flags(PyObject* o, const char* name, const at::Device& dev, int64_t B) {
    const Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kBool) is(t, name, at::kByte, dev, 1);
    is(t, name, t.scalar_type(), dev, 1);
    dense(t, name);
    if (t.size(0) != B) value_error(std::string(name) + " must be [B]");
    return static_cast<const uint8_t*>(t.data_ptr());
}
// A contiguous int32 array of n elements (n < 0: any number).
int32_t* ints(PyObject* o, const char* name, const at::Device& dev, int64_t n) {
    const Tensor& t = tensor(o, name);
    is(t, name, at::kInt, dev, 1);
    dense(t, name);
    if (n >= 0 && t.size(0) != n) value_error(std::string(name) + " must be [" + std::to_string(n) + "]");
    return static_cast<int32_t*>(t.data_ptr());
}
const Tensor& table_of(PyObject* o, const at::Device& dev, int64_t B) {
    const Tensor& t = tensor(o, "block_table");
    is(t, "block_table", at::kInt, dev, 2);
    if (t.size(0) != B || (t.size(1) > 1 && t.stride(1) != 1))
        value_error("block_table must be [B, max_pages] with contiguous rows");
    return t;
}
PyObject* tuple_of(std::initializer_list<Tensor> parts) {
    PyObject* r = PyTuple_New((Py_ssize_t)parts.size());
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (const Tensor& t : parts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

// q, k_cache, v_cache, shared_pages, shared_len, block_table, seq_lens, shares,
// scale, k_scale, v_scale, workspace, out, return_lse, lse
PyObject* shared_prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k_cache"), &v = tensor(a[2], "v_cache");
        const int dt = half_code(q, "q");
        const at::ScalarType type = q.scalar_type();
        const at::Device dev = q.device();
        heads(q, "q", type, dev, -1, 0, 0);
        const int64_t B = q.size(0), Hq = q.size(1), D = q.size(2);
        const Caches c = caches(k, v, type, dev, D, number(a[9]), number(a[10]));
        const int32_t* shared = ints(a[3], "shared_pages", dev, -1);
        const Tensor& table = table_of(a[5], dev, B);
        const int32_t* lens = ints(a[6], "seq_lens", dev, B);
        const uint8_t* shares = a[7] == Py_None ? nullptr : flags(a[7], "shares", dev, B);
        const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)D) : number(a[8]);
        const OnDevice on(dev);
        Tensor ws;
        if (a[11] == Py_None) {
            size_t bytes = 0;
            check("moe_shared_prefix_workspace_bytes",
                  moe_shared_prefix_workspace_bytes(size32(B, "q"), size32(Hq, "q"), c.heads, size32(D, "q"), &bytes));
            ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
            ws.narrow(0, 0, MOE_ATTN_COUNTER_BYTES).zero_();
        } else {
            ws = tensor(a[11], "workspace");
            is(ws, "workspace", at::kByte, dev, 1);
            dense(ws, "workspace");
        }
        const Tensor out = output(a[12], "out", {B, Hq, D}, q.options());
        const bool want = truth(a[13]);
        Tensor lse;
        if (want || a[14] != Py_None) lse = output(a[14], "lse", {B, Hq}, q.options().dtype(at::kFloat));
        check("moe_shared_prefix_attention",
              moe_shared_prefix_attention(
                  q.data_ptr(), step_of(q, 0), step_of(q, 1), size32(B, "q"), size32(Hq, "q"), c.heads, size32(D, "q"), dt,
                  c.k, c.v, c.dtype, c.pages, c.page, shared, size32(THPVariable_Unpack(a[3]).size(0), "shared_pages"),
                  integer(a[4]), shares, static_cast<const int32_t*>(table.data_ptr()), step_of(table, 0),
                  size32(table.size(1), "block_table"), lens, (float)scale, ws.data_ptr(), (size_t)ws.numel(), out.data_ptr(),
                  lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr, on.stream));
        return want ? tuple_of({out, lse}) : THPVariable_Wrap(out);
    });
}

// logits, k, bias, score, groups, top_groups, group_score, renormalize, scale,
// topk_ids, topk_w
PyObject* router_grouped_topk(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 11, [&]() -> PyObject* {
        const Tensor& logits = tensor(a[0], "logits");
        const at::ScalarType type = logits.scalar_type();
        if (type != at::kFloat && type != at::kBFloat16 && type != at::kHalf)
            type_error(std::string("logits must be float32, bfloat16 or float16, got ") + c10::toString(type));
        const at::Device dev = logits.device();
        is(logits, "logits", type, dev, 2);
        last_dense(logits, "logits");
        const int64_t T = logits.size(0), E = logits.size(1);
        const int k = integer(a[1]);
        if (k < 0) value_error("k must not be negative");
        const float* bias = nullptr;
        if (a[2] != Py_None) {
            const Tensor& b = tensor(a[2], "bias");
            is(b, "bias", at::kFloat, dev, 1);
            dense(b, "bias");
            if (b.size(0) != E) value_error("bias must be [E]");
            bias = static_cast<const float*>(b.data_ptr());
        }
        const OnDevice on(dev);
        const Tensor ids = output(a[9], "topk_ids", {T, k}, logits.options().dtype(at::kInt));
        const Tensor w = output(a[10], "topk_w", {T, k}, logits.options().dtype(at::kFloat));
        check("moe_router_grouped_topk",
              moe_router_grouped_topk(logits.data_ptr(), step_of(logits, 0), size32(T, "logits"), size32(E, "logits"),
                                      dtype_code(type), bias, k, integer(a[3]), integer(a[4]), integer(a[5]), integer(a[6]),
                                      truth(a[7]) ? 1 : 0, (float)number(a[8]), static_cast<int32_t*>(ids.data_ptr()),
                                      static_cast<float*>(w.data_ptr()), on.stream));
        return tuple_of({ids, w});
    });
}

// past_lens, new_lens, block_table, free_pages, n_free, page_size, tokens,
// shared_pages, shares, positions, slots, seq_ids, starts, seq_lens, n_free_out
PyObject* plan_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 15, [&]() -> PyObject* {
        const Tensor& past = tensor(a[0], "past_lens");
        const at::Device dev = past.device();
        is(past, "past_lens", at::kInt, dev, 1);
        dense(past, "past_lens");
        const int64_t B = past.size(0);
        const int32_t* news = ints(a[1], "new_lens", dev, B);
        const Tensor& table = table_of(a[2], dev, B);
        const int32_t* stack = ints(a[3], "free_pages", dev, -1);
        const int32_t* height = ints(a[4], "n_free", dev, 1);
        const int T = integer(a[6]);
        if (T < 0) value_error("tokens must not be negative");
        int64_t ns = 0;
        const int32_t* shared = nullptr;
        if (a[7] != Py_None) {
            shared = ints(a[7], "shared_pages", dev, -1);
            ns = THPVariable_Unpack(a[7]).size(0);
        }
        const uint8_t* shares = a[8] == Py_None ? nullptr : flags(a[8], "shares", dev, B);
        const OnDevice on(dev);
        const at::TensorOptions i32 = past.options();
        const Tensor pos = output(a[9], "positions", {T}, i32), slots = output(a[10], "slots", {T}, i32.dtype(at::kLong)),
                     seqs = output(a[11], "seq_ids", {T}, i32), starts = output(a[12], "starts", {B + 1}, i32),
                     lens = output(a[13], "seq_lens", {B}, i32), left = output(a[14], "n_free_out", {1}, i32);
        auto p32 = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
        check("moe_plan_pages",
              moe_plan_pages(p32(past), news, size32(B, "past_lens"), p32(table), step_of(table, 0),
                             size32(table.size(1), "block_table"), stack, size32(THPVariable_Unpack(a[3]).size(0), "free_pages"),
                             height, integer(a[5]), shared, size32(ns, "shared_pages"), shares, T, p32(pos),
                             static_cast<int64_t*>(slots.data_ptr()), p32(seqs), p32(starts), p32(lens), p32(left), on.stream));
        return tuple_of({pos, slots, seqs, starts, lens, left});
    });
}

// block_table, seq_lens, ended, free_pages, n_free, page_size, shared, shares,
// seq_lens_out, n_free_out
PyObject* release_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
    return guarded(n, 10, [&]() -> PyObject* {
        const Tensor& past = tensor(a[1], "seq_lens");
        const at::Device dev = past.device();
        is(past, "seq_lens", at::kInt, dev, 1);
        dense(past, "seq_lens");
        const int64_t B = past.size(0);
        const Tensor& table = table_of(a[0], dev, B);
        const uint8_t* ended = flags(a[2], "ended", dev, B);
        int32_t* stack = ints(a[3], "free_pages", dev, -1);
        const int32_t* height = ints(a[4], "n_free", dev, 1);
        const uint8_t* shares = a[7] == Py_None ? nullptr : flags(a[7], "shares", dev, B);
        const OnDevice on(dev);
        const Tensor lens = output(a[8], "seq_lens_out", {B}, past.options()), left = output(a[9], "n_free_out", {1}, past.options());
        auto p32 = [](const Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); };
        check("moe_release_pages",
              moe_release_pages(p32(table), step_of(table, 0), size32(table.size(1), "block_table"), p32(past),
                                size32(B, "seq_lens"), ended, stack, size32(THPVariable_Unpack(a[3]).size(0), "free_pages"),
                                height, integer(a[5]), integer(a[6]), shares, p32(lens), p32(left), on.stream));
        return tuple_of({lens, left});
    });
}

PyObject* set_fail(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(g_fail, f);
    Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"set_fail", set_fail, METH_O, "callable (function, status) that raises"},
    {"paged_attention", fast(paged_attention), METH_FASTCALL, nullptr},
    {"rope_append", fast(rope_append), METH_FASTCALL, nullptr},
    {"norm_residual", fast(norm_residual), METH_FASTCALL, nullptr},
    {"matvec4", fast(matvec4), METH_FASTCALL, nullptr},
    {"shared_prefix_attention", fast(shared_prefix_attention), METH_FASTCALL, nullptr},
    {"router_grouped_topk", fast(router_grouped_topk), METH_FASTCALL, nullptr},
    {"plan_pages", fast(plan_pages), METH_FASTCALL, nullptr},
    {"release_pages", fast(release_pages), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block(void) { return PyModule_Create(&module); }
