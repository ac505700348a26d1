// binding.cpp -- the Python module _binding: argument marshalling of the rotary, verification and
// commit entry points (include/infllmv2.h).  A serving loop makes these calls once per layer or step
// on a few rows, where the kernels take 2 to 4 us: a call through ctypes, with its checks of types, shapes
// and strides in Python, took 15 to 20 us of host time, one through this module 3.0 to 3.3.
//
// Each function takes the tensors of the Python function of its name (infllmv2.py, which documents
// them) by position, raises ValueError for a tensor of another type, shape or place, and returns the
// entry point's status.  The call is made on the tensors' device, on its current stream unless one is
// given.
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string.h>

#include <new>
#include <sstream>
#include <stdexcept>
#include <string>

#include "infllmv2.h"

namespace {

using at::ScalarType;
using Shape = c10::IntArrayRef;

struct Bad : std::runtime_error {  // becomes a ValueError
    using std::runtime_error::runtime_error;
};

[[noreturn]] void bad(const std::string& text) { throw Bad(text); }

// A call's tensors: all on one CUDA device.
struct Call {
    c10::Device dev{c10::DeviceType::CPU};
    bool seen = false;
    const at::Tensor* all[16];
    int count = 0;

    const at::Tensor& tensor(PyObject* o, const char* name) {
        if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
        const at::Tensor& t = THPVariable_Unpack(o);
        all[count++] = &t;  // at most 12 of a call
        return t;
    }
    const at::Tensor* maybe(PyObject* o, const char* name) { return o == Py_None ? nullptr : &tensor(o, name); }
    void place() {  // after the checks of types and shapes
        for (int i = 0; i < count; ++i) {
            const c10::Device d = all[i]->device();
            if (!seen) {
                if (!d.is_cuda()) bad("tensor must live on a CUDA device");
                dev = d;
                seen = true;
            } else if (d != dev) {
                bad("all tensors must live on one device");
            }
        }
    }
};

std::string text(Shape s) {
    std::ostringstream o;
    o << s;
    return o.str();
}

// Type, shape and density of a tensor that a call reads or writes whole.
void want(const char* name, const at::Tensor& t, Shape shape, ScalarType type, ScalarType other = ScalarType::Undefined) {
    const ScalarType s = t.scalar_type();
    if ((s == type || s == other) && t.sizes() == shape && t.is_contiguous()) return;
    bad(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor of shape " + text(shape));
}

struct Rows {
    int64_t heads, ld;
};
// [*lead, heads, d] with dense heads and one stride between rows, as a slice of a fused projection has.
Rows head_rows(const char* name, const at::Tensor& t, Shape lead, ScalarType type, int64_t d) {
    const Shape s = t.sizes(), st = t.strides();
    const size_t n = lead.size();
    if (t.scalar_type() != type || s.size() != n + 2 || s.slice(0, n) != lead || s[n + 1] != d)
        bad(std::string(name) + " must be a " + c10::toString(type) + " tensor of shape " + text(lead) + " + [heads, " +
            std::to_string(d) + "]");
    const int64_t H = s[n], width = H * d;
    bool ok = st[n + 1] == 1 && (H == 1 || st[n] == d);
    int64_t ld = width;
    if (n == 1) {
        if (lead[0] > 1) ld = st[0];
    } else {
        ld = lead[1] > 1 ? st[1] : lead[0] > 1 ? st[0] : width;
        ok = ok && (lead[0] <= 1 || lead[1] == 0 || st[0] == ld * lead[1]);
    }
    if (t.numel() > 0 && !(ok && ld >= width)) bad(std::string(name) + " must have dense heads and evenly spaced rows");
    return {H, ld < width ? width : ld};
}

int as_int(int64_t x, const char* name) {
    if (x < INT32_MIN || x > INT32_MAX) bad(std::string(name) + " is out of range");
    return static_cast<int>(x);
}

int64_t integer(PyObject* o) {
    const int64_t x = PyLong_AsLongLong(o);
    if (x == -1 && PyErr_Occurred()) throw std::runtime_error("");  // Python's error is set
    return x;
}

// A parameter structure: its ctypes object (by the buffer protocol), or a dict of its fields.
template <typename P>
bool from_buffer(PyObject* o, P* p) {
    if (PyDict_Check(o) || !PyObject_CheckBuffer(o)) return false;
    Py_buffer b;
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw std::runtime_error("");
    const bool fits = b.len == sizeof(P);
    if (fits) memcpy(p, b.buf, sizeof(P));
    PyBuffer_Release(&b);
    if (!fits) bad("not a parameter structure of this call");
    return true;
}
// The names of the fields, made once.
struct Names {
    PyObject* key[11];
    Names() {
        const char* const text[11] = {"rotary_dim", "interleaved", "attn_scale", "block_size", "kernel_size", "kernel_stride",
                                      "topk", "n_init_blocks", "n_local_blocks", "dense_len", "softmax_scale"};
        for (int i = 0; i < 11; ++i) key[i] = PyUnicode_InternFromString(text[i]);
    }
};
enum : int {
    kRotaryDim, kInterleaved, kAttnScale, kBlockSize, kKernelSize, kKernelStride, kTopk, kNInit, kNLocal, kDenseLen,
    kSoftmaxScale
};
PyObject* field(PyObject* o, int which, bool needed) {  // new reference, or nullptr
    static const Names names;
    PyObject* const key = names.key[which];
    if (key == nullptr) throw std::bad_alloc();
    if (PyDict_CheckExact(o)) {
        PyObject* v = PyDict_GetItemWithError(o, key);
        if (v != nullptr) return Py_NewRef(v);
        if (PyErr_Occurred()) throw std::runtime_error("");
        if (needed) {
            PyErr_SetObject(PyExc_KeyError, key);
            throw std::runtime_error("");
        }
        return nullptr;
    }
    PyObject* v = PyObject_GetItem(o, key);
    if (v == nullptr) {
        if (needed || !PyErr_ExceptionMatches(PyExc_KeyError)) throw std::runtime_error("");
        PyErr_Clear();
    }
    return v;
}
// A field as Python's int() and float() take it.
int32_t int_field(PyObject* o, int which, bool needed = true) {
    PyObject* v = field(o, which, needed);
    if (v == nullptr) return 0;
    PyObject* i = PyLong_CheckExact(v) ? Py_NewRef(v) : PyNumber_Long(v);
    Py_DECREF(v);
    if (i == nullptr) throw std::runtime_error("");
    const int64_t x = PyLong_AsLongLong(i);
    Py_DECREF(i);
    if (x == -1 && PyErr_Occurred()) throw std::runtime_error("");
    return as_int(x, "a parameter");
}
float float_field(PyObject* o, int which) {
    PyObject* v = field(o, which, false);
    if (v == nullptr) return 0.f;
    const double x = PyFloat_AsDouble(v);
    Py_DECREF(v);
    if (x == -1.0 && PyErr_Occurred()) throw std::runtime_error("");
    return static_cast<float>(x);
}
infllmv2_rope_params rope_params(PyObject* o) {
    infllmv2_rope_params p;
    if (from_buffer(o, &p)) return p;
    p.rotary_dim = int_field(o, kRotaryDim);
    p.interleaved = int_field(o, kInterleaved, false);
    p.attn_scale = float_field(o, kAttnScale);
    return p;
}
infllmv2_params method_params(PyObject* o) {
    infllmv2_params p;
    if (from_buffer(o, &p)) return p;
    p.block_size = int_field(o, kBlockSize);
    p.kernel_size = int_field(o, kKernelSize);
    p.kernel_stride = int_field(o, kKernelStride);
    p.topk = int_field(o, kTopk);
    p.n_init_blocks = int_field(o, kNInit);
    p.n_local_blocks = int_field(o, kNLocal);
    p.dense_len = int_field(o, kDenseLen);
    p.softmax_scale = float_field(o, kSoftmaxScale);
    return p;
}

// Calls f(stream) on the tensors' device.
template <typename F>
PyObject* enqueue(Call& call, PyObject* stream, F f) {
    call.place();
    const c10::cuda::OptionalCUDAGuard guard(call.dev);
    void* s;
    if (stream == Py_None) {
        s = c10::cuda::getCurrentCUDAStream(call.dev.index()).stream();
    } else if (PyLong_Check(stream)) {
        s = PyLong_AsVoidPtr(stream);
    } else {
        PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
        if (h == nullptr) throw std::runtime_error("");
        s = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
    }
    if (PyErr_Occurred()) throw std::runtime_error("");
    return PyLong_FromLong(f(s));
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t expected, F f) {
    try {
        if (n != expected) bad("wrong number of arguments");
        return f();
    } catch (const Bad& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

template <typename T = void>
T* ptr(const at::Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* ptr(const at::Tensor* t) {
    return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr());
}
int dtype_of(const at::Tensor& t, const char* name) {
    if (t.scalar_type() == ScalarType::Float) return INFLLMV2_FP32;
    if (t.scalar_type() == ScalarType::BFloat16) return INFLLMV2_BF16;
    bad(std::string(name) + " must be bf16 or fp32");
}
void check_dim(const char* name, const at::Tensor& t, int64_t n) {
    if (t.dim() != n) bad(std::string(name) + " must have " + std::to_string(n) + " dimensions");
}
void check_freqs(const at::Tensor& freqs, const infllmv2_rope_params& rp) {
    want("freqs", freqs, {rp.rotary_dim / 2}, ScalarType::Long, ScalarType::UInt64);
}

// q, k, pos, q_out, k_out, freqs, rope, transposed, stream
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded(na, 9, [&]() -> PyObject* {
        Call call;
        const at::Tensor& q = call.tensor(a[0], "q");
        const at::Tensor* k = call.maybe(a[1], "k");
        const at::Tensor& pos = call.tensor(a[2], "pos");
        const at::Tensor& qo = call.tensor(a[3], "q_out");
        const at::Tensor* ko = call.maybe(a[4], "k_out");
        const at::Tensor& freqs = call.tensor(a[5], "freqs");
        const infllmv2_rope_params rp = rope_params(a[6]);
        const int transposed = PyObject_IsTrue(a[7]);
        if (transposed < 0) throw std::runtime_error("");
        check_dim("q", q, 3);
        if ((k == nullptr) != (ko == nullptr)) bad("k and k_out must be given together");
        const int type = dtype_of(q, "q");
        const int64_t rows = q.size(0), d = q.size(2);
        const Shape lead = q.sizes().slice(0, 1);
        const Rows rq = head_rows("q", q, lead, q.scalar_type(), d), rqo = head_rows("q_out", qo, lead, q.scalar_type(), d);
        Rows rk{0, 0}, rko{0, 0};
        if (k != nullptr) {
            rk = head_rows("k", *k, lead, q.scalar_type(), d);
            rko = head_rows("k_out", *ko, lead, q.scalar_type(), d);
        }
        if (rq.heads != rqo.heads || rk.heads != rko.heads) bad("outputs must have their inputs' heads");
        want("pos", pos, lead, ScalarType::Int);
        check_freqs(freqs, rp);
        return enqueue(call, a[8], [&](void* s) {
            return infllmv2_rope(ptr(q), rq.ld, ptr(k), rk.ld, ptr<int32_t>(pos), ptr<uint64_t>(freqs), as_int(rows, "rows"),
                                 as_int(rq.heads, "heads"), as_int(rk.heads, "heads"), as_int(d, "d"), type, transposed,
                                 ptr(qo), rqo.ld, ptr(ko), rko.ld, &rp, s);
        });
    });
}

struct Chunk {
    int B, Tq, total;
};
// Sizes of a chunk call with rows of leading sizes `lead`: [B, Tq] without cu_q, [total_q] with it.
Chunk chunk(Shape lead, int64_t B, const at::Tensor* cu_q, PyObject* Tq_max, const at::Tensor& kv_len,
            const at::Tensor& freqs, const infllmv2_rope_params& rp) {
    want("kv_len", kv_len, {B}, ScalarType::Int);
    check_freqs(freqs, rp);
    if (cu_q == nullptr) {
        if (lead.size() != 2 || lead[0] != B) bad("rows must be [B, Tq, heads, d] without cu_q");
        return {as_int(B, "B"), as_int(lead[1], "Tq"), as_int(B * lead[1], "rows")};
    }
    if (lead.size() != 1 || Tq_max == Py_None) bad("rows must be [total_q, heads, d] with cu_q, and Tq_max be given");
    want("cu_q", *cu_q, {B + 1}, ScalarType::Int);
    return {as_int(B, "B"), as_int(integer(Tq_max), "Tq_max"), as_int(lead[0], "rows")};
}

// q, k_new, v_new, q_out, k_cache, v_cache, kv_len, freqs, rope, cu_q, Tq_max, stream
PyObject* py_rope_append(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded(na, 12, [&]() -> PyObject* {
        Call call;
        const at::Tensor &q = call.tensor(a[0], "q"), &k = call.tensor(a[1], "k_new"), &v = call.tensor(a[2], "v_new"),
                         &qo = call.tensor(a[3], "q_out"), &kc = call.tensor(a[4], "k_cache"),
                         &vc = call.tensor(a[5], "v_cache"), &kv_len = call.tensor(a[6], "kv_len"),
                         &freqs = call.tensor(a[7], "freqs");
        const infllmv2_rope_params rp = rope_params(a[8]);
        const at::Tensor* cu_q = call.maybe(a[9], "cu_q");
        constexpr ScalarType bf16 = ScalarType::BFloat16;
        check_dim("k_cache", kc, 4);
        if (q.dim() < 2) bad("q must have heads of d elements");
        const int64_t B = kc.size(0), Hkv = kc.size(1), L_max = kc.size(2), d = kc.size(3);
        const Shape lead = q.sizes().slice(0, q.dim() - 2);
        const Chunk ch = chunk(lead, B, cu_q, a[10], kv_len, freqs, rp);
        const Rows rq = head_rows("q", q, lead, bf16, d), rk = head_rows("k_new", k, lead, bf16, d),
                   rv = head_rows("v_new", v, lead, bf16, d);
        if (rk.heads != Hkv || rv.heads != Hkv) bad("k_new and v_new must have the caches' heads");
        want("q_out", qo, q.sizes(), bf16);
        want("k_cache", kc, {B, Hkv, L_max, d}, bf16);
        want("v_cache", vc, {B, Hkv, L_max, d}, bf16);
        return enqueue(call, a[11], [&](void* s) {
            return infllmv2_rope_append(ptr(q), rq.ld, ptr(k), rk.ld, ptr(v), rv.ld, ptr(qo), ptr(kc), ptr(vc),
                                        ptr<int32_t>(kv_len), ptr<int32_t>(cu_q), ptr<uint64_t>(freqs), ch.B, ch.Tq, ch.total,
                                        as_int(rq.heads, "heads"), as_int(Hkv, "heads"), as_int(d, "d"),
                                        as_int(L_max, "L_max"), &rp, s);
        });
    });
}

// dq, dk, dv, dq_out, dk_out, dv_out, kv_len, freqs, rope, cu_q, Tq_max, stream
PyObject* py_rope_append_bwd(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded(na, 12, [&]() -> PyObject* {
        Call call;
        const at::Tensor &dq = call.tensor(a[0], "dq"), &dk = call.tensor(a[1], "dk"), &dv = call.tensor(a[2], "dv"),
                         &dqo = call.tensor(a[3], "dq_out"), &dko = call.tensor(a[4], "dk_out"),
                         &dvo = call.tensor(a[5], "dv_out"), &kv_len = call.tensor(a[6], "kv_len"),
                         &freqs = call.tensor(a[7], "freqs");
        const infllmv2_rope_params rp = rope_params(a[8]);
        const at::Tensor* cu_q = call.maybe(a[9], "cu_q");
        constexpr ScalarType f32 = ScalarType::Float;
        check_dim("dk", dk, 4);
        if (dq.dim() < 2) bad("dq must have heads of d elements");
        const int64_t B = dk.size(0), Hkv = dk.size(1), L_max = dk.size(2), d = dk.size(3);
        const Shape lead = dq.sizes().slice(0, dq.dim() - 2);
        const Chunk ch = chunk(lead, B, cu_q, a[10], kv_len, freqs, rp);
        const int type = dtype_of(dqo, "dq_out");
        const ScalarType t = dqo.scalar_type();
        const Rows rq = head_rows("dq_out", dqo, lead, t, d), rk = head_rows("dk_out", dko, lead, t, d),
                   rv = head_rows("dv_out", dvo, lead, t, d);
        if (rk.heads != Hkv || rv.heads != Hkv) bad("dk_out and dv_out must have the caches' heads");
        want("dq", dq, dqo.sizes(), f32);
        want("dk", dk, {B, Hkv, L_max, d}, f32);
        want("dv", dv, {B, Hkv, L_max, d}, f32);
        return enqueue(call, a[11], [&](void* s) {
            return infllmv2_rope_append_bwd(ptr<float>(dq), ptr<float>(dk), ptr<float>(dv), ptr(dqo), rq.ld, ptr(dko), rk.ld,
                                            ptr(dvo), rv.ld, ptr<int32_t>(kv_len), ptr<int32_t>(cu_q), ptr<uint64_t>(freqs),
                                            ch.B, ch.Tq, ch.total, as_int(rq.heads, "heads"), as_int(Hkv, "heads"),
                                            as_int(d, "d"), as_int(L_max, "L_max"), type, &rp, s);
        });
    });
}

// q, k_new, v_new, q_out, draft_k, draft_v, kv_len, tree_mask, freqs, rope, stream
PyObject* py_rope_drafts(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded(na, 11, [&]() -> PyObject* {
        Call call;
        const at::Tensor &q = call.tensor(a[0], "q"), &k = call.tensor(a[1], "k_new"), &v = call.tensor(a[2], "v_new"),
                         &qo = call.tensor(a[3], "q_out"), &dk = call.tensor(a[4], "draft_k"),
                         &dv = call.tensor(a[5], "draft_v"), &kv_len = call.tensor(a[6], "kv_len"),
                         &mask = call.tensor(a[7], "tree_mask"), &freqs = call.tensor(a[8], "freqs");
        const infllmv2_rope_params rp = rope_params(a[9]);
        constexpr ScalarType bf16 = ScalarType::BFloat16;
        check_dim("draft_k", dk, 4);
        const int64_t B = dk.size(0), Hkv = dk.size(1), n = dk.size(2), d = dk.size(3);
        const int64_t lead_[2] = {B, n};
        const Shape lead(lead_, 2);
        const Rows rq = head_rows("q", q, lead, bf16, d), rk = head_rows("k_new", k, lead, bf16, d),
                   rv = head_rows("v_new", v, lead, bf16, d);
        if (rk.heads != Hkv || rv.heads != Hkv) bad("k_new and v_new must have the draft buffers' heads");
        want("q_out", qo, q.sizes(), bf16);
        want("draft_k", dk, {B, Hkv, n, d}, bf16);
        want("draft_v", dv, {B, Hkv, n, d}, bf16);
        want("kv_len", kv_len, {B}, ScalarType::Int);
        want("tree_mask", mask, lead, ScalarType::Long, ScalarType::UInt64);
        check_freqs(freqs, rp);
        return enqueue(call, a[10], [&](void* s) {
            return infllmv2_rope_drafts(ptr(q), rq.ld, ptr(k), rk.ld, ptr(v), rv.ld, ptr(qo), ptr(dk), ptr(dv),
                                        ptr<int32_t>(kv_len), ptr<uint64_t>(mask), ptr<uint64_t>(freqs), as_int(B, "B"),
                                        as_int(n, "n_draft"), as_int(rq.heads, "heads"), as_int(Hkv, "heads"), as_int(d, "d"),
                                        &rp, s);
        });
    });
}

// tokens, target, draft, u, path, n_path, out_tokens, tree_mask, n_nodes, kv_len, kv_len_out, replace, stream
PyObject* py_verify(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded(na, 13, [&]() -> PyObject* {
        Call call;
        const at::Tensor &tokens = call.tensor(a[0], "tokens"), &target = call.tensor(a[1], "target");
        const at::Tensor* draft = call.maybe(a[2], "draft");
        const at::Tensor &u = call.tensor(a[3], "u"), &path = call.tensor(a[4], "path"),
                         &n_path = call.tensor(a[5], "n_path"), &out = call.tensor(a[6], "out_tokens");
        const at::Tensor *mask = call.maybe(a[7], "tree_mask"), *nodes = call.maybe(a[8], "n_nodes"),
                         *kv = call.maybe(a[9], "kv_len"), *kvo = call.maybe(a[10], "kv_len_out");
        const int replace = PyObject_IsTrue(a[11]);
        if (replace < 0) throw std::runtime_error("");
        check_dim("tokens", tokens, 2);
        check_dim("target", target, 3);
        const int64_t B = tokens.size(0), n = tokens.size(1), V = target.size(2);
        const Shape bn = tokens.sizes();
        constexpr ScalarType i32 = ScalarType::Int;
        const int type = dtype_of(target, "target");
        want("tokens", tokens, bn, i32);
        want("target", target, {B, n, V}, target.scalar_type());
        if (draft != nullptr) want("draft", *draft, {B, n, V}, target.scalar_type());
        want("u", u, bn, ScalarType::Float);
        want("path", path, bn, i32);
        want("n_path", n_path, {B}, i32);
        want("out_tokens", out, bn, i32);
        if (mask != nullptr) want("tree_mask", *mask, bn, ScalarType::Long, ScalarType::UInt64);
        if (nodes != nullptr) want("n_nodes", *nodes, {B}, i32);
        if ((kv == nullptr) != (kvo == nullptr)) bad("kv_len and kv_len_out must be given together");
        if (kv != nullptr) {
            want("kv_len", *kv, {B}, i32);
            want("kv_len_out", *kvo, {B}, i32);
        }
        return enqueue(call, a[12], [&](void* s) {
            return infllmv2_verify(ptr<int32_t>(tokens), ptr<uint64_t>(mask), ptr<int32_t>(nodes), ptr(target), ptr(draft),
                                   ptr<float>(u), ptr<int32_t>(kv), as_int(B, "B"), as_int(n, "n_draft"), as_int(V, "V"), type,
                                   replace, ptr<int32_t>(path), ptr<int32_t>(n_path), ptr<int32_t>(out), ptr<int32_t>(kvo), s);
        });
    });
}

// draft_k, draft_v, path, n_path, k_cache, v_cache, kernel_cache, kv_len, params, stream
PyObject* py_commit(PyObject*, PyObject* const* a, Py_ssize_t na) {
    return guarded(na, 10, [&]() -> PyObject* {
        Call call;
        const at::Tensor &dk = call.tensor(a[0], "draft_k"), &dv = call.tensor(a[1], "draft_v"),
                         &path = call.tensor(a[2], "path"), &n_path = call.tensor(a[3], "n_path"),
                         &kc = call.tensor(a[4], "k_cache"), &vc = call.tensor(a[5], "v_cache");
        const at::Tensor* kern = call.maybe(a[6], "kernel_cache");
        const at::Tensor& kv_len = call.tensor(a[7], "kv_len");
        const infllmv2_params p = method_params(a[8]);
        constexpr ScalarType bf16 = ScalarType::BFloat16, i32 = ScalarType::Int;
        check_dim("draft_k", dk, 4);
        check_dim("k_cache", kc, 4);
        const int64_t B = dk.size(0), Hkv = dk.size(1), n = dk.size(2), d = dk.size(3), L_max = kc.size(2);
        if (kern != nullptr) check_dim("kernel_cache", *kern, 4);
        const int64_t M_max = kern == nullptr ? 0 : kern->size(2);
        want("draft_k", dk, {B, Hkv, n, d}, bf16);
        want("draft_v", dv, {B, Hkv, n, d}, bf16);
        want("path", path, {B, n}, i32);
        want("n_path", n_path, {B}, i32);
        want("k_cache", kc, {B, Hkv, L_max, d}, bf16);
        want("v_cache", vc, {B, Hkv, L_max, d}, bf16);
        if (kern != nullptr) want("kernel_cache", *kern, {B, Hkv, M_max, d}, bf16);
        want("kv_len", kv_len, {B}, i32);
        return enqueue(call, a[9], [&](void* s) {
            return infllmv2_commit(ptr(dk), ptr(dv), ptr<int32_t>(path), ptr<int32_t>(n_path), ptr(kc), ptr(vc), ptr(kern),
                                   ptr<int32_t>(kv_len), as_int(B, "B"), as_int(n, "n_draft"), as_int(Hkv, "heads"),
                                   as_int(d, "d"), as_int(L_max, "L_max"), as_int(M_max, "M_max"), &p, s);
        });
    });
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Fast f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method("rope", py_rope),
                           method("rope_append", py_rope_append),
                           method("rope_append_bwd", py_rope_append_bwd),
                           method("rope_drafts", py_rope_drafts),
                           method("verify", py_verify),
                           method("commit", py_commit),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&g_module); }
