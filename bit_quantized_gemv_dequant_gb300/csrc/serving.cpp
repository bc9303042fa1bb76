// Python module _serving: the serving operators' calls on torch tensors. It
// marshals arguments to the C ABI as the ctypes binding does for the other
// calls: checks of tensors, new outputs, the current stream, scratch. Written
// against the CPython and ATen headers because that is most of a short call's
// time: the two calls of an fp8 projection of one token took 25 us of host time
// through ctypes, of which the two launches are 7.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <map>
#include <mutex>
#include <optional>
#include <string>
#include <utility>

#include "qgemv.h"

namespace {

using at::ScalarType;
using at::Tensor;

PyObject* g_error = nullptr;  // QGError

struct Raised {};  // a Python exception is set

template <class... A>
[[noreturn]] void value_error(const char* format, A... args) {
    PyErr_Format(PyExc_ValueError, format, args...);
    throw Raised{};
}

void check(int status, const char* what) {
    if (status == QG_OK) return;
    if (PyObject* e = PyObject_CallFunction(g_error, "si", what, status)) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw Raised{};
}

const Tensor& cuda(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) value_error("%s must be a CUDA tensor", name);
    const Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) value_error("%s must be a CUDA tensor", name);
    return t;
}

const Tensor& dense(PyObject* o, const char* name) {
    const Tensor& t = cuda(o, name);
    if (!t.is_contiguous()) value_error("%s must be contiguous", name);
    return t;
}

const Tensor& dense(PyObject* o, const char* name, ScalarType type) {
    const Tensor& t = dense(o, name);
    if (t.scalar_type() != type) value_error("%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    return t;
}

void dims(const Tensor& t, const char* name, int64_t n) {
    if (t.dim() != n) value_error("%s must have %lld dimensions, got %lld", name, (long long)n, (long long)t.dim());
}

void shape(const Tensor& t, const char* name, at::IntArrayRef want) {
    if (t.sizes().equals(want)) return;
    std::string w, g;
    for (int64_t n : want) w += (w.empty() ? "" : ", ") + std::to_string(n);
    for (int64_t n : t.sizes()) g += (g.empty() ? "" : ", ") + std::to_string(n);
    value_error("%s must have the shape (%s), got (%s)", name, w.c_str(), g.c_str());
}

// A tensor whose rows t[i] are dense; the rows may lie apart.
const Tensor& rows(PyObject* o, const char* name, int64_t n, int64_t* stride) {
    const Tensor& t = cuda(o, name);
    dims(t, name, n);
    int64_t step = 1;
    for (int64_t i = n - 1; i > 0; --i) {
        if (t.size(i) > 1 && t.stride(i) != step && t.numel() > 0) value_error("%s must have dense rows", name);
        step *= t.size(i);
    }
    *stride = t.size(0) > 1 && t.numel() > 0 ? t.stride(0) : step;
    return t;
}

int code(const Tensor& t, const char* name) {
    switch (t.scalar_type()) {
        case ScalarType::Float: return QG_F32;
        case ScalarType::Half: return QG_F16;
        case ScalarType::BFloat16: return QG_BF16;
        default: value_error("%s must be float32, float16 or bfloat16, got %s", name, c10::toString(t.scalar_type()));
    }
}

Tensor make(at::IntArrayRef size, ScalarType type, const Tensor& like) {
    return at::empty(size, at::TensorOptions().dtype(type).device(like.device()));
}

template <class T = void>
T* at_of(const Tensor& t) {
    return static_cast<T*>(t.data_ptr());
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw Raised{};
    return v;
}

bool truth(PyObject* o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v != 0;
}

qg_stream_t stream_of(PyObject* o) {
    if (o == Py_None) return reinterpret_cast<qg_stream_t>(c10::cuda::getCurrentCUDAStream().stream());
    PyObject* v = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
    if (!v) throw Raised{};
    void* p = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    if (!p && PyErr_Occurred()) throw Raised{};
    return reinterpret_cast<qg_stream_t>(p);
}

// The caller's workspace, or a buffer of this (device, stream) that grows on
// demand: calls on different streams may run at the same time and must not
// share one. On one stream the kernels of a call that pass data through it must
// not have another call's between them, hence a mutex for each, held while a call
// enqueues. A call that is being captured gets a buffer of its own, from the
// graph's memory: the graph may run on any stream, beside other graphs. The map
// is guarded by the interpreter's lock; never destroyed, as the process may end
// after CUDA has.
struct Held {
    Tensor buffer;
    std::mutex enqueue;
};
struct Scratch {
    Tensor owner;  // another thread may grow the buffer before this call is enqueued
    void* p = nullptr;
    size_t n = 0;
    std::mutex* enqueue = nullptr;
};
Scratch scratch(size_t need, PyObject* workspace, const Tensor& like, qg_stream_t s) {
    if (workspace != Py_None) {
        const Tensor& t = dense(workspace, "workspace");
        return {t, t.data_ptr(), (size_t)t.nbytes()};
    }
    if (need == 0) return {};
    cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(reinterpret_cast<cudaStream_t>(s), &status) != cudaSuccess) {
        // the legacy stream, while another one is captured: it is not itself
        (void)cudaGetLastError();
        status = cudaStreamCaptureStatusNone;
    }
    if (status != cudaStreamCaptureStatusNone) {
        const Tensor t = make({(int64_t)need}, ScalarType::Byte, like);
        return {t, t.data_ptr(), need};
    }
    static auto* held = new std::map<std::pair<int, qg_stream_t>, Held>;
    Held& h = (*held)[{like.get_device(), s}];
    if (!h.buffer.defined() || (size_t)h.buffer.numel() < need) h.buffer = make({(int64_t)need}, ScalarType::Byte, like);
    return {h.buffer, h.buffer.data_ptr(), (size_t)h.buffer.numel(), &h.enqueue};
}

// The interpreter's lock is released while one of these lives, and taken again
// however its scope is left.
class Unlocked {
  public:
    Unlocked() : state_(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(state_); }
    Unlocked(const Unlocked&) = delete;
    Unlocked& operator=(const Unlocked&) = delete;

  private:
    PyThreadState* state_;
};

// The library's call, without the interpreter's lock but with the scratch's. f
// may throw: it asks tensors for their data, which those under a transform do not
// give.
template <class F>
void call(const char* what, std::mutex* enqueue, F&& f) {
    int status;
    {
        const Unlocked unlocked;
        std::unique_lock<std::mutex> alone;
        if (enqueue) alone = std::unique_lock<std::mutex>(*enqueue);
        status = f();
    }
    check(status, what);
}
template <class F>
void call(const char* what, F&& f) {
    call(what, nullptr, std::forward<F>(f));
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }

template <class... T>
PyObject* tuple(const T&... t) {
    PyObject* r = PyTuple_New(sizeof...(T));
    if (!r) throw Raised{};
    Py_ssize_t i = 0;
    for (PyObject* o : {wrap(t)...}) PyTuple_SET_ITEM(r, i++, o);
    return r;
}

// A Python function of N arguments, the last one the stream, exceptions turned
// into Python's. With a stream given the call is as under torch.cuda.stream(it):
// new outputs and scratch belong to it, so that no work still under way on the
// current stream has to do with their memory.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
        return nullptr;
    }
    try {
        std::optional<c10::cuda::CUDAStreamGuard> guard;
        if (N > 1 && a[N - 1] != Py_None)
            guard.emplace(c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(stream_of(a[N - 1])),
                                                           c10::cuda::current_device()));
        return F(a);
    } catch (const Raised&) {
        return nullptr;
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
        return nullptr;
    }
}

// ------------------------------------------------------------------- the calls
PyObject* set_error(PyObject* const* a) {
    Py_XDECREF(g_error);
    g_error = Py_NewRef(a[0]);
    Py_RETURN_NONE;
}

// x, codes | None, scales | None, stream
PyObject* quantize_fp8_b128(PyObject* const* a) {
    int64_t stride;
    const Tensor& x = rows(a[0], "x", 2, &stride);
    const int type = code(x, "x");
    const int64_t M = x.size(0), K = x.size(1), KB = (K + 127) / 128;
    const Tensor codes = a[1] == Py_None ? make({M, K}, ScalarType::Float8_e4m3fn, x)
                                         : dense(a[1], "codes", ScalarType::Float8_e4m3fn);
    const Tensor scales = a[2] == Py_None ? make({M, KB}, ScalarType::Float, x) : dense(a[2], "scales", ScalarType::Float);
    if (a[1] != Py_None) shape(codes, "codes", {M, K});
    if (a[2] != Py_None) shape(scales, "scales", {M, KB});
    const qg_stream_t s = stream_of(a[3]);
    call("quantize_fp8_b128", [&] {
        return ::quantize_fp8_b128(x.data_ptr(), type, stride, at_of<uint8_t>(codes), at_of<float>(scales), M, K, s);
    });
    return tuple(codes, scales);
}

// a, a_scales, w, w_scales, y | None, out_dtype, workspace, stream
PyObject* qmm_fp8_b128(PyObject* const* a) {
    const Tensor& x = dense(a[0], "a", ScalarType::Float8_e4m3fn);
    const Tensor& sx = dense(a[1], "a_scales", ScalarType::Float);
    const Tensor& w = dense(a[2], "w", ScalarType::Float8_e4m3fn);
    const Tensor& sw = dense(a[3], "w_scales", ScalarType::Float);
    dims(x, "a", 2);
    dims(w, "w", 2);
    const int64_t M = x.size(0), K = x.size(1), N = w.size(0), KB = (K + 127) / 128;
    shape(w, "w", {N, K});
    shape(sx, "a_scales", {M, KB});
    shape(sw, "w_scales", {(N + 127) / 128, KB});
    if (a[4] == Py_None && !THPDtype_Check(a[5])) value_error("out_dtype must be a torch.dtype");
    const Tensor y = a[4] == Py_None ? make({M, N}, reinterpret_cast<THPDtype*>(a[5])->scalar_type, x) : dense(a[4], "y");
    if (a[4] != Py_None) shape(y, "y", {M, N});
    const int type = code(y, "y");
    const qg_stream_t s = stream_of(a[7]);
    size_t need = 0;
    const uintptr_t odd = (uintptr_t)K | (uintptr_t)x.data_ptr() | (uintptr_t)w.data_ptr();
    if (odd & 15) check(qmm_fp8_b128_workspace_size(M, N, K, &need), "qmm_fp8_b128");
    const Scratch ws = scratch(need, a[6], x, s);
    call("qmm_fp8_b128", ws.enqueue, [&] {
        return ::qmm_fp8_b128(at_of<uint8_t>(x), at_of<float>(sx), at_of<uint8_t>(w), at_of<float>(sw), y.data_ptr(), type,
                              M, N, K, ws.p, ws.n, s);
    });
    return wrap(y);
}

// q, k_cache, v_cache, page_table, q_offsets, context_lens, out | None, lse | None,
// max_new | None, scale | None, softcap, window, return_lse, workspace, stream
PyObject* attn_paged(PyObject* const* a) {
    int64_t stride;
    const Tensor& q = rows(a[0], "q", 3, &stride);
    const ScalarType type = q.scalar_type();
    const int dtype = code(q, "q");
    const Tensor& k = dense(a[1], "k_cache", type);
    const Tensor& v = dense(a[2], "v_cache", type);
    const Tensor& table = dense(a[3], "page_table", ScalarType::Int);
    const Tensor& offsets = dense(a[4], "q_offsets", ScalarType::Int);
    const Tensor& lens = dense(a[5], "context_lens", ScalarType::Int);
    const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2);
    dims(k, "k_cache", 4);
    dims(table, "page_table", 2);
    const int64_t pages = k.size(0), Hkv = k.size(1), page = k.size(2), B = table.size(0);
    shape(k, "k_cache", {pages, Hkv, page, D});
    shape(v, "v_cache", {pages, Hkv, page, D});
    shape(offsets, "q_offsets", {B + 1});
    shape(lens, "context_lens", {B});
    const Tensor out = a[6] == Py_None ? make({T, Hq, D}, type, q) : dense(a[6], "out", type);
    if (a[6] != Py_None) shape(out, "out", {T, Hq, D});
    Tensor lse;
    if (a[7] != Py_None) {
        lse = dense(a[7], "lse", ScalarType::Float);
        shape(lse, "lse", {T, Hq});
    } else if (truth(a[12])) {
        lse = make({T, Hq}, ScalarType::Float, q);
    }
    const int64_t max_new = a[8] == Py_None ? T : integer(a[8]);
    const float scale = a[9] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(a[9]);
    const float softcap = (float)number(a[10]);
    const int64_t window = integer(a[11]);
    const qg_stream_t s = stream_of(a[14]);
    size_t need = 0;
    check(attn_paged_workspace_size(T, B, max_new, Hq, Hkv, D, &need), "attn_paged");
    const Scratch ws = scratch(need, a[13], q, s);
    call("attn_paged", ws.enqueue, [&] {
        return ::attn_paged(q.data_ptr(), stride, k.data_ptr(), v.data_ptr(), at_of<int32_t>(table), at_of<int32_t>(offsets),
                            at_of<int32_t>(lens), out.data_ptr(), lse.defined() ? at_of<float>(lse) : nullptr, dtype, T, B,
                            max_new, Hq, Hkv, D, pages, page, table.size(1), scale, softcap, window, ws.p, ws.n, s);
    });
    return lse.defined() ? tuple(out, lse) : wrap(out);
}

// k, v, k_cache, v_cache, slots, stream
PyObject* kv_append(PyObject* const* a) {
    int64_t ks, vs;
    const Tensor& k = rows(a[0], "k", 3, &ks);
    const Tensor& v = rows(a[1], "v", 3, &vs);
    const Tensor& kc = dense(a[2], "k_cache");
    const Tensor& vc = dense(a[3], "v_cache", kc.scalar_type());
    const Tensor& slots = dense(a[4], "slots", ScalarType::Long);
    if (v.scalar_type() != k.scalar_type()) value_error("k and v must be of one type");
    dims(kc, "k_cache", 4);
    const int64_t T = k.size(0), H = k.size(1), D = k.size(2), pages = kc.size(0), page = kc.size(2);
    shape(v, "v", {T, H, D});
    shape(kc, "k_cache", {pages, H, page, D});
    shape(vc, "v_cache", {pages, H, page, D});
    shape(slots, "slots", {T});
    const int x = code(k, "k"), c = code(kc, "k_cache");
    const qg_stream_t s = stream_of(a[5]);
    call("kv_append", [&] {
        return ::kv_append(k.data_ptr(), v.data_ptr(), ks, vs, x, kc.data_ptr(), vc.data_ptr(), c, at_of<int64_t>(slots), T, H,
                           D, pages, page, s);
    });
    Py_RETURN_NONE;
}

struct Planes {
    void* cache;
    int64_t planes, pages, bytes;
};
Planes planes(PyObject* o) {
    const Tensor& t = dense(o, "cache");
    if (t.dim() < 3 || t.numel() == 0) value_error("cache must be [planes, num_pages, ...] with at least one value");
    const int64_t n = t.size(0), pages = t.size(1);
    return {t.data_ptr(), n, pages, t.numel() / (n * pages) * t.element_size()};
}

// cache, src, dst, stream
PyObject* kv_copy_pages(PyObject* const* a) {
    const Planes p = planes(a[0]);
    const Tensor& src = dense(a[1], "src", ScalarType::Int);
    const Tensor& dst = dense(a[2], "dst", ScalarType::Int);
    shape(dst, "dst", src.sizes());
    const qg_stream_t s = stream_of(a[3]);
    call("kv_copy_pages", [&] {
        return ::kv_copy_pages(p.cache, p.planes, p.pages, p.bytes, at_of<int32_t>(src), at_of<int32_t>(dst), src.numel(), s);
    });
    Py_RETURN_NONE;
}

// cache, page_table, lens, ref_counts, parents, page_size, workspace, stream
PyObject* kv_fork(PyObject* const* a) {
    const Planes p = planes(a[0]);
    const Tensor& table = dense(a[1], "page_table", ScalarType::Int);
    const Tensor& lens = dense(a[2], "lens", ScalarType::Int);
    const Tensor& refs = dense(a[3], "ref_counts", ScalarType::Int);
    const Tensor& parents = dense(a[4], "parents", ScalarType::Int);
    dims(table, "page_table", 2);
    const int64_t R = table.size(0), W = table.size(1), n = parents.numel();
    shape(lens, "lens", {R});
    shape(refs, "ref_counts", {p.pages});
    const int64_t page_size = integer(a[5]);
    const Tensor ct = make({n, W}, ScalarType::Int, table), cl = make({n}, ScalarType::Int, table);
    const Tensor nr = make({p.pages}, ScalarType::Int, table);
    const qg_stream_t s = stream_of(a[7]);
    size_t need = 0;
    check(kv_fork_workspace_size(n, &need), "kv_fork");
    const Scratch ws = scratch(need, a[6], table, s);
    call("kv_fork", ws.enqueue, [&] {
        return ::kv_fork(p.cache, p.planes, p.pages, p.bytes, page_size, at_of<int32_t>(table), at_of<int32_t>(lens),
                         at_of<int32_t>(refs), R, W, at_of<int32_t>(parents), n, at_of<int32_t>(ct), at_of<int32_t>(cl),
                         at_of<int32_t>(nr), ws.p, ws.n, s);
    });
    return tuple(ct, cl, nr);
}

// page_table, lens, ref_counts, drop, stream
PyObject* kv_free(PyObject* const* a) {
    const Tensor& table = dense(a[0], "page_table", ScalarType::Int);
    const Tensor& lens = dense(a[1], "lens", ScalarType::Int);
    const Tensor& refs = dense(a[2], "ref_counts", ScalarType::Int);
    const Tensor& drop = dense(a[3], "drop", ScalarType::Byte);
    dims(table, "page_table", 2);
    const int64_t R = table.size(0), W = table.size(1), pages = refs.numel();
    shape(lens, "lens", {R});
    shape(drop, "drop", {R});
    shape(refs, "ref_counts", {pages});
    const Tensor nt = make({R, W}, ScalarType::Int, table), nl = make({R}, ScalarType::Int, table);
    const Tensor nr = make({pages}, ScalarType::Int, table);
    const qg_stream_t s = stream_of(a[4]);
    call("kv_free", [&] {
        return ::kv_free(at_of<int32_t>(table), at_of<int32_t>(lens), at_of<int32_t>(refs), at_of<uint8_t>(drop), R, W, pages,
                         at_of<int32_t>(nt), at_of<int32_t>(nl), at_of<int32_t>(nr), s);
    });
    return tuple(nt, nl, nr);
}

// cache, page_table, ref_counts, workspace, stream
PyObject* kv_compact(PyObject* const* a) {
    const Planes p = planes(a[0]);
    const Tensor& table = dense(a[1], "page_table", ScalarType::Int);
    const Tensor& refs = dense(a[2], "ref_counts", ScalarType::Int);
    dims(table, "page_table", 2);
    const int64_t R = table.size(0), W = table.size(1);
    shape(refs, "ref_counts", {p.pages});
    const Tensor nt = make({R, W}, ScalarType::Int, table), nr = make({p.pages}, ScalarType::Int, table);
    const Tensor map = make({p.pages}, ScalarType::Int, table), live = make({1}, ScalarType::Int, table);
    const qg_stream_t s = stream_of(a[4]);
    size_t need = 0;
    check(kv_compact_workspace_size(p.pages, &need), "kv_compact");
    const Scratch ws = scratch(need, a[3], table, s);
    call("kv_compact", ws.enqueue, [&] {
        return ::kv_compact(p.cache, p.planes, p.pages, p.bytes, at_of<int32_t>(table), R, W, at_of<int32_t>(refs),
                            at_of<int32_t>(nt), at_of<int32_t>(nr), at_of<int32_t>(map), at_of<int32_t>(live), ws.p, ws.n, s);
    });
    return tuple(nt, nr, map, live);
}

// logits, targets, top_k, stream
PyObject* token_logprobs(PyObject* const* a) {
    int64_t stride;
    const Tensor& x = rows(a[0], "logits", 2, &stride);
    const int type = code(x, "logits");
    const Tensor& targets = dense(a[1], "targets", ScalarType::Long);
    const int64_t M = x.size(0), V = x.size(1), k = std::min(integer(a[2]), V);
    shape(targets, "targets", {M});
    const Tensor lp = make({M}, ScalarType::Float, x), h = make({M}, ScalarType::Float, x);
    const Tensor r = make({M}, ScalarType::Int, x);
    const Tensor tv = make({M, std::max<int64_t>(k, 0)}, ScalarType::Float, x);
    const Tensor ti = make({M, std::max<int64_t>(k, 0)}, ScalarType::Int, x);
    const qg_stream_t s = stream_of(a[3]);
    call("token_logprobs", [&] {
        return ::token_logprobs(x.data_ptr(), type, stride, at_of<int64_t>(targets), M, V,
                                (int)std::max<int64_t>(std::min<int64_t>(k, 1 << 20), -1), at_of<float>(lp), at_of<float>(h),
                                at_of<int32_t>(r), at_of<float>(tv), at_of<int32_t>(ti), s);
    });
    return tuple(lp, h, r, tv, ti);
}

#define ENTRY(name, n) {#name, (PyCFunction)(void*)entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {ENTRY(set_error, 1),     ENTRY(quantize_fp8_b128, 4), ENTRY(qmm_fp8_b128, 8),
                           ENTRY(attn_paged, 15),   ENTRY(kv_append, 6),         ENTRY(kv_copy_pages, 4),
                           ENTRY(kv_fork, 8),       ENTRY(kv_free, 5),           ENTRY(kv_compact, 5),
                           ENTRY(token_logprobs, 4), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() { return PyModule_Create(&g_module); }
