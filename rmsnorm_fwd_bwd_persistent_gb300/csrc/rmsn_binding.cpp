// rmsn_binding.cpp -- the tensor side of the entry points qk_norm_rope_* and kv4_* as a CPython
// module: checks shapes, dtypes, devices and strides, allocates the outputs and workspaces that
// the caller did not pass, and calls the C ABI on the current stream of the tensors' device.
//
// Compiled, because these calls stand before kernels of a few microseconds: the same checks and
// packing written in Python took 12 to 20 us per call on the Grace host, the kernels of a decoding
// step 4 to 8.  Every function returns its tensors, or the library's status as an int if it is
// not 0 (the Python wrappers raise it); wrong arguments raise TypeError or ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdio>
#include <initializer_list>
#include <optional>
#include <string>
#include <utility>

#include "rmsn.h"

namespace {

using at::Tensor;

constexpr int64_t kBlock = 16;  // tokens per record of the cache

// A refused argument: the Python exception to raise, and its text.
struct Refused {
    PyObject* type;
    std::string text;
};
struct AlreadySet {};  // the interpreter has the exception

template <typename... A>
Refused refused(PyObject* type, const char* format, A... a) {
    char text[512];
    std::snprintf(text, sizeof text, format, a...);
    return {type, text};
}
inline Refused refused(PyObject* type, const char* text) { return {type, text}; }

template <typename... A>
Refused TypeError(A... a) {
    return refused(PyExc_TypeError, a...);
}
template <typename... A>
Refused ValueError(A... a) {
    return refused(PyExc_ValueError, a...);
}

const Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) throw TypeError("%s must be a torch.Tensor", name);
    return THPVariable_Unpack(o);
}

struct Named {
    const Tensor& t;
    const char* name;
};

// The CUDA device of all the tensors.
int device_of(std::initializer_list<Named> ts) {
    for (const Named& n : ts)
        if (!n.t.is_cuda())
            throw ValueError("%s must be a CUDA tensor (got %s)", n.name, n.t.device().str().c_str());
    const int dev = ts.begin()->t.get_device();
    for (const Named& n : ts)
        if (n.t.get_device() != dev)
            throw ValueError("%s is on cuda:%d, %s on cuda:%d", n.name, (int)n.t.get_device(),
                             ts.begin()->name, dev);
    return dev;
}

int dtype_code(const Tensor& t, const char* name) {
    if (t.scalar_type() == at::kFloat) return RMSN_F32;
    if (t.scalar_type() == at::kBFloat16) return RMSN_BF16;
    throw TypeError("%s: unsupported dtype (float32 or bfloat16)", name);
}

rmsn_heads_t heads(const Tensor& t, const char* name) {
    const int64_t n = t.dim();
    if (t.stride(n - 1) != 1 && t.size(n - 1) > 1 && t.numel() > 0)
        throw ValueError("%s: the elements of a head must be next to each other", name);
    return {t.data_ptr(), n == 4 ? t.stride(0) : 0, t.stride(n - 3), t.stride(n - 2), t.size(n - 2)};
}

struct Rows {
    int64_t B, T, D;
};

Rows rows(const Tensor& q, const Tensor& k, bool batched) {
    const int64_t n = q.dim();
    if (k.dim() != n || !(n == 3 || (n == 4 && batched)))
        throw ValueError(batched ? "q and k must be [T, heads, D] or [B, S, heads, D]"
                                 : "q and k must be [T, heads, D]");
    if (q.size(-1) != k.size(-1) || q.size(n - 3) != k.size(n - 3) || q.size(0) != k.size(0))
        throw ValueError("q and k must have the same tokens and the same head size");
    if (q.scalar_type() != k.scalar_type()) throw TypeError("q and k must be of one dtype");
    return {n == 4 ? q.size(0) : 1, q.size(n - 3), q.size(-1)};
}

int weights(const Tensor& wq, const Tensor& wk, int64_t D) {
    for (const Tensor* w : {&wq, &wk})
        if (w->dim() != 1 || w->size(0) != D || !w->is_contiguous())
            throw ValueError("wq and wk must be a contiguous [%lld]", (long long)D);
    if (wq.scalar_type() != wk.scalar_type()) throw TypeError("wq and wk must be of one dtype");
    return dtype_code(wq, "wq");
}

rmsn_rope_t rope(const Tensor& cos, const Tensor& sin, const Tensor& pos, bool neighbours, Rows r,
                 bool batched) {
    if (cos.dim() != 2 || cos.sizes() != sin.sizes())
        throw ValueError("cos and sin must be [positions, rotated dims / 2]");
    if (cos.scalar_type() != at::kFloat || sin.scalar_type() != at::kFloat)
        throw TypeError("cos and sin must be float32");
    if (!cos.is_contiguous() || !sin.is_contiguous())
        throw ValueError("cos and sin must be contiguous");
    if (pos.scalar_type() != at::kLong) throw TypeError("positions must be int64");
    rmsn_rope_t p{static_cast<const float*>(cos.data_ptr()), static_cast<const float*>(sin.data_ptr()),
                  cos.size(0), 2 * cos.size(1), neighbours,
                  static_cast<const int64_t*>(pos.data_ptr()), 0, 0};
    if (pos.dim() == 1 && pos.size(0) == r.T) {
        p.pos_token_stride = pos.stride(0);
    } else if (batched && pos.dim() == 2 && pos.size(0) == r.B && pos.size(1) == r.T) {
        p.pos_batch_stride = pos.stride(0);
        p.pos_token_stride = pos.stride(1);
    } else {
        throw ValueError("positions must be [T] (or [B, S] beside q of [B, S, heads, D])");
    }
    return p;
}

// A new contiguous tensor beside another (straight from the allocator: the dispatcher costs as much
// again).
Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const Tensor& like) {
    return Tensor(at::detail::empty_cuda(shape, type, like.device(), std::nullopt));
}

// A caller's output, checked, or a new contiguous one.
Tensor output(PyObject* o, at::IntArrayRef shape, at::ScalarType type, const Tensor& like,
              const char* name, bool contiguous) {
    if (o == Py_None) return fresh(shape, type, like);
    const Tensor& t = tensor(o, name);
    device_of({{like, "the input"}, {t, name}});
    if (t.sizes() != shape || t.scalar_type() != type || (contiguous && !t.is_contiguous()))
        throw ValueError("%s must have the expected shape and dtype%s", name,
                         contiguous ? " and be contiguous" : "");
    return t;
}

Tensor scratch(PyObject* o, size_t need, const Tensor& like) {
    if (o == Py_None)
        return fresh({(int64_t)(need < 16 ? 16 : need)}, at::kByte, like);
    const Tensor& t = tensor(o, "workspace");
    device_of({{like, "the input"}, {t, "workspace"}});
    if (!t.is_contiguous()) throw ValueError("workspace must be contiguous");
    return t;
}

size_t bytes(const Tensor& t) { return (size_t)t.numel() * t.element_size(); }

void arguments(Py_ssize_t got, Py_ssize_t want) {
    if (got != want) throw TypeError("%d arguments expected, got %d", (int)want, (int)got);
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw AlreadySet{};
    return v;
}

int64_t integer(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw AlreadySet{};
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw AlreadySet{};
    return v != 0;
}

// Calls the library on the device's current stream without the interpreter's lock.
template <typename F>
int enqueue(int dev, F call) {
    const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
    const auto stream = reinterpret_cast<rmsn_stream_t>(
        c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = call(stream);
    Py_END_ALLOW_THREADS
    return status;
}

// The tensors as a tuple (an object that the caller passed comes back itself), or the status.
PyObject* result(int status, std::initializer_list<std::pair<PyObject*, const Tensor*>> outs) {
    if (status != RMSN_OK) return PyLong_FromLong(status);
    PyObject* tuple = PyTuple_New((Py_ssize_t)outs.size());
    if (!tuple) throw AlreadySet{};
    Py_ssize_t i = 0;
    for (const auto& o : outs) {
        PyObject* item = o.first == Py_None ? THPVariable_Wrap(*o.second) : Py_NewRef(o.first);
        if (!item) {
            Py_DECREF(tuple);
            throw AlreadySet{};
        }
        PyTuple_SET_ITEM(tuple, i++, item);
    }
    return tuple;
}

// q, k, wq, wk, cos, sin, positions, eps, interleaved, q_out, k_out
PyObject* fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    arguments(n, 11);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &wq = tensor(a[2], "wq"),
                 &wk = tensor(a[3], "wk"), &cos = tensor(a[4], "cos"), &sin = tensor(a[5], "sin"),
                 &pos = tensor(a[6], "positions");
    const int dev = device_of({{q, "q"}, {k, "k"}, {wq, "wq"}, {wk, "wk"}, {cos, "cos"},
                               {sin, "sin"}, {pos, "positions"}});
    const Rows r = rows(q, k, true);
    const int wd = weights(wq, wk, r.D), xd = dtype_code(q, "q");
    const rmsn_rope_t rp = rope(cos, sin, pos, truth(a[8]), r, q.dim() == 4);
    const float eps = (float)number(a[7]);
    const Tensor yq = output(a[9], q.sizes(), q.scalar_type(), q, "q_out", false);
    const Tensor yk = output(a[10], k.sizes(), k.scalar_type(), k, "k_out", false);
    const rmsn_heads_t hq = heads(q, "q"), hk = heads(k, "k"), oq = heads(yq, "q_out"),
                       ok = heads(yk, "k_out");
    const int st = enqueue(dev, [&](rmsn_stream_t s) {
        return qk_norm_rope_fwd(&hq, &hk, xd, wq.data_ptr(), wk.data_ptr(), wd, &rp, &oq, &ok, r.B,
                                r.T, r.D, eps, s);
    });
    return result(st, {{a[9], &yq}, {a[10], &yk}});
}

// gq, gk, q, k, wq, wk, cos, sin, positions, eps, interleaved, workspace, dq, dk, dwq, dwk
PyObject* bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    arguments(n, 16);
    const Tensor &gq = tensor(a[0], "gq"), &gk = tensor(a[1], "gk"), &q = tensor(a[2], "q"),
                 &k = tensor(a[3], "k"), &wq = tensor(a[4], "wq"), &wk = tensor(a[5], "wk"),
                 &cos = tensor(a[6], "cos"), &sin = tensor(a[7], "sin"),
                 &pos = tensor(a[8], "positions");
    const int dev = device_of({{gq, "gq"}, {gk, "gk"}, {q, "q"}, {k, "k"}, {wq, "wq"}, {wk, "wk"},
                               {cos, "cos"}, {sin, "sin"}, {pos, "positions"}});
    const Rows r = rows(q, k, true);
    if (gq.sizes() != q.sizes() || gk.sizes() != k.sizes() ||
        gq.scalar_type() != q.scalar_type() || gk.scalar_type() != k.scalar_type())
        throw ValueError("gq and gk must have the shapes and dtype of q and k");
    const int wd = weights(wq, wk, r.D), xd = dtype_code(q, "q");
    const rmsn_rope_t rp = rope(cos, sin, pos, truth(a[10]), r, q.dim() == 4);
    const float eps = (float)number(a[9]);
    const Tensor dq = output(a[12], q.sizes(), q.scalar_type(), q, "dq", false);
    const Tensor dk = output(a[13], k.sizes(), k.scalar_type(), k, "dk", false);
    const Tensor dwq = output(a[14], {r.D}, at::kFloat, q, "dwq", true);
    const Tensor dwk = output(a[15], {r.D}, at::kFloat, q, "dwk", true);
    const Tensor ws = scratch(a[11], qk_norm_rope_bwd_workspace_bytes(r.D, dev), q);
    const rmsn_heads_t hq = heads(q, "q"), hk = heads(k, "k"), yq = heads(gq, "gq"),
                       yk = heads(gk, "gk"), oq = heads(dq, "dq"), ok = heads(dk, "dk");
    const int st = enqueue(dev, [&](rmsn_stream_t s) {
        return qk_norm_rope_bwd(&yq, &yk, &hq, &hk, xd, wq.data_ptr(), wk.data_ptr(), wd, &rp, &oq, &ok,
                                static_cast<float*>(dwq.data_ptr()), static_cast<float*>(dwk.data_ptr()),
                                r.B, r.T, r.D, eps, ws.data_ptr(), bytes(ws), s);
    });
    return result(st, {{a[12], &dq}, {a[13], &dk}, {a[14], &dwq}, {a[15], &dwk}});
}

struct Cache {
    rmsn_kv4_t c;
    int64_t D;
};

Cache cache_of(const Tensor& t) {
    if (t.dim() != 4 || t.scalar_type() != at::kByte || !t.is_contiguous() || t.size(3) % 20)
        throw ValueError("cache must be a contiguous uint8 tensor of kv4_cache_shape(...)");
    return {{t.data_ptr(), t.size(0), t.size(1), t.size(2) * kBlock}, t.size(3) / 20};
}

const int64_t* slots_of(const Tensor& t, int64_t T) {
    if (t.scalar_type() != at::kLong || t.dim() != 1 || !t.is_contiguous() || t.size(0) != T)
        throw ValueError("slots must be a contiguous int64 [T]");
    return static_cast<const int64_t*>(t.data_ptr());
}

// q, k, v, wq, wk, cos, sin, positions, cache, slots, eps, interleaved, q_out
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    arguments(n, 13);
    const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
                 &wq = tensor(a[3], "wq"), &wk = tensor(a[4], "wk"), &cos = tensor(a[5], "cos"),
                 &sin = tensor(a[6], "sin"), &pos = tensor(a[7], "positions"),
                 &cache = tensor(a[8], "cache"), &slots = tensor(a[9], "slots");
    const int dev = device_of({{q, "q"}, {k, "k"}, {v, "v"}, {wq, "wq"}, {wk, "wk"}, {cos, "cos"},
                               {sin, "sin"}, {pos, "positions"}, {cache, "cache"}, {slots, "slots"}});
    const Rows r = rows(q, k, false);
    if (q.scalar_type() != at::kBFloat16 || v.scalar_type() != at::kBFloat16)
        throw TypeError("q, k and v must be bfloat16");
    if (v.sizes() != k.sizes()) throw ValueError("v must have k's shape");
    const int wd = weights(wq, wk, r.D);
    const rmsn_rope_t rp = rope(cos, sin, pos, truth(a[11]), r, false);
    const float eps = (float)number(a[10]);
    const Cache c = cache_of(cache);
    if (c.D != r.D || c.c.kv_heads != k.size(1)) throw ValueError("the cache is for other heads than k");
    const int64_t* sl = slots_of(slots, r.T);
    const Tensor y = output(a[12], q.sizes(), q.scalar_type(), q, "q_out", false);
    const rmsn_heads_t hq = heads(q, "q"), hk = heads(k, "k"), hv = heads(v, "v"), o = heads(y, "q_out");
    const int st = enqueue(dev, [&](rmsn_stream_t s) {
        return qk_norm_rope_kv4_append(&hq, &hk, &hv, wq.data_ptr(), wk.data_ptr(), wd, &rp, &o, &c.c, sl,
                                       r.T, r.D, eps, s);
    });
    return result(st, {{a[12], &y}});
}

// cache, slots, k, v
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
    arguments(n, 4);
    const Tensor &cache = tensor(a[0], "cache"), &slots = tensor(a[1], "slots");
    const int dev = device_of({{cache, "cache"}, {slots, "slots"}});
    const Cache c = cache_of(cache);
    const int64_t T = slots.dim() == 1 ? slots.size(0) : -1;
    const int64_t* sl = slots_of(slots, T);
    const Tensor k = output(a[2], {T, c.c.kv_heads, c.D}, at::kBFloat16, cache, "k", false);
    const Tensor v = output(a[3], {T, c.c.kv_heads, c.D}, at::kBFloat16, cache, "v", false);
    const rmsn_heads_t hk = heads(k, "k"), hv = heads(v, "v");
    const int st = enqueue(dev, [&](rmsn_stream_t s) {
        return kv4_read(&c.c, sl, &hk, &hv, T, c.D, s);
    });
    return result(st, {{a[2], &k}, {a[3], &v}});
}

// q, cache, page_table, kv_lens, cu_q, max_q, scale, out, lse, workspace
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
    arguments(n, 10);
    const Tensor &q = tensor(a[0], "q"), &cache = tensor(a[1], "cache"),
                 &table = tensor(a[2], "page_table"), &lens = tensor(a[3], "kv_lens");
    const int dev = device_of({{q, "q"}, {cache, "cache"}, {table, "page_table"}, {lens, "kv_lens"}});
    if (q.dim() != 3 || q.scalar_type() != at::kBFloat16)
        throw ValueError("q must be bfloat16 [T, heads, D]");
    const Cache c = cache_of(cache);
    const int64_t T = q.size(0), H = q.size(1);
    if (q.size(2) != c.D || c.c.kv_heads < 1 || H % c.c.kv_heads != 0)
        throw ValueError("the cache is for other heads than q");
    if (table.scalar_type() != at::kInt || table.dim() != 2 ||
        (table.size(1) > 1 && table.stride(1) != 1))
        throw ValueError("page_table must be int32 [seqs, width] with unit stride in the width");
    const int64_t seqs = table.size(0), width = table.size(1);
    if (lens.scalar_type() != at::kInt || lens.dim() != 1 || lens.size(0) != seqs || !lens.is_contiguous())
        throw ValueError("kv_lens must be a contiguous int32 [seqs]");
    const int32_t* cu = nullptr;
    if (a[4] == Py_None) {
        if (T != seqs) throw ValueError("without cu_q there is one query token per sequence");
    } else {
        const Tensor& t = tensor(a[4], "cu_q");
        device_of({{q, "q"}, {t, "cu_q"}});
        if (t.scalar_type() != at::kInt || t.dim() != 1 || t.size(0) != seqs + 1 || !t.is_contiguous())
            throw ValueError("cu_q must be a contiguous int32 [seqs + 1]");
        cu = static_cast<const int32_t*>(t.data_ptr());
    }
    const int64_t max_q = integer(a[5]);
    const float scale = a[6] == Py_None ? (float)(1.0 / std::sqrt((double)c.D)) : (float)number(a[6]);
    const Tensor o = output(a[7], q.sizes(), at::kBFloat16, q, "out", false);
    const Tensor lse = output(a[8], {T, H}, at::kFloat, q, "lse", true);
    const Tensor ws = scratch(a[9], kv4_attention_workspace_bytes(seqs, c.D, dev), q);
    const rmsn_heads_t hq = heads(q, "q"), ho = heads(o, "out");
    const int st = enqueue(dev, [&](rmsn_stream_t s) {
        return kv4_attention(&hq, &c.c, static_cast<const int32_t*>(table.data_ptr()), width,
                             seqs > 1 ? table.stride(0) : width, static_cast<const int32_t*>(lens.data_ptr()),
                             cu, max_q, seqs, T, c.D, scale, &ho, static_cast<float*>(lse.data_ptr()),
                             ws.data_ptr(), bytes(ws), s);
    });
    return result(st, {{a[7], &o}, {a[8], &lse}});
}

using Function = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);

// No C++ exception leaves the module: refusals as above, torch's own (out of memory, ...) by its
// translation.
template <Function F>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    try {
        return F(self, a, n);
    } catch (const Refused& e) {
        PyErr_SetString(e.type, e.text.c_str());
        return nullptr;
    } catch (const AlreadySet&) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

PyMethodDef method(const char* name, Function f) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method("qk_norm_rope_fwd", guarded<fwd>),
                          method("qk_norm_rope_bwd", guarded<bwd>),
                          method("qk_norm_rope_kv4_append", guarded<append>),
                          method("kv4_read", guarded<read>),
                          method("kv4_attention", guarded<attention>),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
