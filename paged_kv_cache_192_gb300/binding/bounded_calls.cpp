// Torch-facing binding of the bounded-cache calls (rotary store, compaction,
// windowed decode and prefill): argument checks, output allocation, and the
// call into the C ABI of include/pa.h.  Marshalling only, as in ops.py, whose
// functions forward here.
//
// Why not ctypes: a decode step's calls run 3 to 12 us on the GPU, and their
// checks and marshalling in Python took 9 to 18 us on the host.
//
// Errors are the ones of ops.py: ValueError for shapes, devices and layouts,
// TypeError for types, and the callable given to set_check (it raises PAError)
// for a status of the library.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <optional>
#include <string>

#include "pa.h"

namespace {

PyObject *g_check = nullptr;  // raises for a status of the library

struct Refusal {  // a Python exception to set
    PyObject *type;
    std::string text;
};
struct Raised {};  // a Python exception is already set

[[noreturn]] void value_error(std::string s) { throw Refusal{PyExc_ValueError, std::move(s)}; }
[[noreturn]] void type_error(std::string s) { throw Refusal{PyExc_TypeError, std::move(s)}; }

std::string shape(std::initializer_list<int64_t> dims) {
    std::string s;
    for (const int64_t d : dims) s += "[" + std::to_string(d) + "]";
    return s;
}

const at::Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) value_error(std::string(name) + " must be a CUDA tensor");
    return THPVariable_Unpack(o);
}

bool sized(const at::Tensor &t, std::initializer_list<int64_t> dims) {
    return t.sizes() == at::IntArrayRef(dims.begin(), dims.size());
}

// A host integer of the C ABI.
int int32_of(int64_t x, const char *name) {
    if (x < INT32_MIN || x > INT32_MAX)
        value_error(std::string(name) + "=" + std::to_string(x) + " does not fit 32 bits");
    return static_cast<int>(x);
}
int int32_of(PyObject *o, const char *name) {
    PyObject *i = PyNumber_Index(o);
    if (!i) throw Raised{};
    int overflow = 0;
    const long long x = PyLong_AsLongLongAndOverflow(i, &overflow);
    Py_DECREF(i);
    if (overflow) value_error(std::string(name) + " does not fit 32 bits");
    return int32_of(static_cast<int64_t>(x), name);
}

float scale_of(PyObject *o, int64_t d) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    const double x = PyFloat_AsDouble(o);
    if (x == -1.0 && PyErr_Occurred()) throw Raised{};
    return static_cast<float>(x);
}

int dtype_of(const at::Tensor &t) {
    if (t.scalar_type() == at::kBFloat16) return PA_BF16;
    if (t.scalar_type() == at::kFloat) return PA_F32;
    type_error(std::string("unsupported dtype ") + c10::toString(t.scalar_type()));
}

// The device and stream of a call: those of its first tensor and the current
// stream there, or the stream given.  Both are current while it lives, so that
// outputs are allocated on the stream that writes them.
struct Place {
    int device;
    std::optional<c10::cuda::CUDAGuard> guard;
    std::optional<c10::cuda::CUDAStreamGuard> on_stream;
    pa_stream_t stream;

    Place(const at::Tensor &first, const char *name, PyObject *given) {
        if (!first.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
        device = first.get_device();
        guard.emplace(static_cast<c10::DeviceIndex>(device));
        if (given != Py_None) {
            const long long dev = attribute(given, "device_index");
            if (dev != device)
                value_error("stream must belong to the tensors' device cuda:" + std::to_string(device));
            on_stream.emplace(c10::cuda::getStreamFromExternal(
                reinterpret_cast<cudaStream_t>(attribute(given, "cuda_stream")),
                static_cast<c10::DeviceIndex>(device)));
        }
        stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
    }
    static long long attribute(PyObject *o, const char *name) {
        PyObject *v = PyObject_GetAttrString(o, name);
        if (!v) throw Raised{};
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred()) throw Raised{};
        return x;
    }
    // address of a tensor of the call
    void *operator()(const at::Tensor &t, const char *name, at::ScalarType type,
                     bool contiguous = true) const {
        if (!t.is_cuda() || t.get_device() != device)
            value_error(std::string(name) + " must be a CUDA tensor on cuda:" + std::to_string(device));
        if (t.scalar_type() != type)
            type_error(std::string(name) + " must be " + c10::toString(type) + ", got " +
                       c10::toString(t.scalar_type()));
        if (contiguous && !t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
        return t.data_ptr();
    }
    at::Tensor new_like(const at::Tensor &t) const {
        return at::Tensor(at::detail::empty_cuda(t.sizes(), t.scalar_type(), t.device(), std::nullopt));
    }
};

// Runs an entry point's body with its positional arguments; exceptions become
// Python's.
template <class F>
PyObject *guarded(const char *what, Py_ssize_t want, Py_ssize_t n, F &&body) {
    HANDLE_TH_ERRORS
    try {
        if (n != want)
            type_error(std::string(what) + " takes " + std::to_string(want) + " arguments, got " +
                       std::to_string(n));
        return body();
    } catch (const Refusal &r) {
        PyErr_SetString(r.type, r.text.c_str());
        return nullptr;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// The library's status; the GIL is released while it launches.
template <class F>
void launch(F &&call) {
    int rc;
    Py_BEGIN_ALLOW_THREADS rc = call();
    Py_END_ALLOW_THREADS if (rc == PA_OK) return;
    PyObject *r = g_check ? PyObject_CallFunction(g_check, "i", rc) : nullptr;
    if (r) {
        Py_DECREF(r);
        PyErr_SetString(PyExc_RuntimeError, "the library's status was not raised");
    } else if (!PyErr_Occurred()) {
        PyErr_SetString(PyExc_RuntimeError, "set_check was not called");
    }
    throw Raised{};
}

// Elements between tokens of [T][H][d] whose heads are contiguous.
int64_t token_rows(const at::Tensor &t, const char *name, int64_t T, int64_t H, int64_t d) {
    if (!sized(t, {T, H, d})) value_error(std::string(name) + " must be " + shape({T, H, d}));
    if (t.stride(2) != 1 || (t.stride(1) != d && H > 1))
        value_error(std::string(name) + ": the heads of a token must be contiguous");
    return T > 1 ? t.stride(0) : H * d;
}

void same_pools(const at::Tensor &k_cache, const at::Tensor &v_cache) {
    if (v_cache.sizes() != k_cache.sizes())
        value_error("k_cache and v_cache must have the same shape");
}

// q, k_new, v_new, k_cache, v_cache, slot_mapping, positions, inv_freq,
// sections, interleaved, q_out, stream
PyObject *rope_reshape_and_cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("rope_reshape_and_cache", 12, n, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &k_new = tensor(a[1], "k_new"),
                         &v_new = tensor(a[2], "v_new"), &k_cache = tensor(a[3], "k_cache"),
                         &v_cache = tensor(a[4], "v_cache"), &slots = tensor(a[5], "slot_mapping"),
                         &positions = tensor(a[6], "positions"), &inv_freq = tensor(a[7], "inv_freq");
        if (q.dim() != 3 || k_new.dim() != 3 || k_cache.dim() != 4)
            value_error("q must be [T][Hq][d], k_new and v_new [T][Hkv][d], pools [NB][Hkv][bs][d]");
        const int64_t NB = k_cache.size(0), Hkv = k_cache.size(1), bs = k_cache.size(2),
                      d = k_cache.size(3), T = q.size(0), Hq = q.size(1);
        same_pools(k_cache, v_cache);
        if (!sized(slots, {T})) value_error("slot_mapping must be " + shape({T}));
        const int64_t axes = positions.dim() == 2 ? positions.size(0) : 1;
        if (!sized(positions, {T}) && !sized(positions, {axes, T}))
            value_error("positions must be " + shape({T}) + " or [axes]" + shape({T}));
        if (inv_freq.dim() != 1) value_error("inv_freq must be [rot/2]");
        const int64_t half = inv_freq.size(0);
        int sections[4] = {int32_of(half, "rot/2"), 0, 0, 0};
        Py_ssize_t nsec = 1;
        if (a[8] != Py_None) {
            PyObject *seq = PySequence_Fast(a[8], "sections must be a sequence");
            if (!seq) throw Raised{};
            struct Drop {
                PyObject *o;
                ~Drop() { Py_DECREF(o); }
            } drop{seq};
            nsec = PySequence_Fast_GET_SIZE(seq);
            if (nsec < 1 || nsec > 4) value_error("sections must name 1 to 4 axes");
            for (Py_ssize_t i = 0; i < nsec; ++i)
                sections[i] = int32_of(PySequence_Fast_GET_ITEM(seq, i), "sections");
        }
        if (nsec != axes)
            value_error("sections must name the frequencies of each of " + std::to_string(axes) + " axes");
        const int inter = PyObject_IsTrue(a[9]);
        if (inter < 0) throw Raised{};
        const int64_t qs = token_rows(q, "q", T, Hq, d), ks = token_rows(k_new, "k_new", T, Hkv, d),
                      vs = token_rows(v_new, "v_new", T, Hkv, d);
        const bool given = a[10] != Py_None;
        const int64_t os = given ? token_rows(tensor(a[10], "q_out"), "q_out", T, Hq, d) : Hq * d;
        const Place place(q, "q", a[11]);
        const at::ScalarType dt = k_cache.scalar_type();
        const int code = dtype_of(k_cache);
        const void *qp = place(q, "q", dt, false), *kp = place(k_new, "k_new", dt, false),
                   *vp = place(v_new, "v_new", dt, false), *fp = place(inv_freq, "inv_freq", at::kFloat),
                   *sp = place(slots, "slot_mapping", at::kLong),
                   *pp = place(positions, "positions", at::kLong);
        void *kc = place(k_cache, "k_cache", dt), *vc = place(v_cache, "v_cache", dt);
        const at::Tensor out = given ? tensor(a[10], "q_out") : place.new_like(q);
        void *op = place(out, "q_out", dt, false);
        const int iT = int32_of(T, "T"), iHq = int32_of(Hq, "Hq"), iHkv = int32_of(Hkv, "Hkv"),
                  ibs = int32_of(bs, "block_size"), id = int32_of(d, "head_dim"),
                  rot = int32_of(2 * half, "rot");
        launch([&] {
            return pa_rope_reshape_and_cache(
                op, os, qp, qs, kp, ks, vp, vs, kc, vc, static_cast<const int64_t *>(sp),
                static_cast<const int64_t *>(pp), static_cast<const float *>(fp), sections,
                static_cast<int>(axes), inter, iT, NB, iHq, iHkv, ibs, id, rot, code, place.stream);
        });
        return THPVariable_Wrap(out);
    });
}

// k_cache, v_cache, src_table, dst_table, keep, keep_lens, stream
PyObject *compact_cache(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("compact_cache", 7, n, [&]() -> PyObject * {
        const at::Tensor &k_cache = tensor(a[0], "k_cache"), &v_cache = tensor(a[1], "v_cache"),
                         &src = tensor(a[2], "src_table"), &dst = tensor(a[3], "dst_table"),
                         &keep = tensor(a[4], "keep"), &keep_lens = tensor(a[5], "keep_lens");
        if (k_cache.dim() != 4) value_error("pools must be [NB][Hkv][bs][d]");
        same_pools(k_cache, v_cache);
        const int64_t Hkv = k_cache.size(1);
        if (keep.dim() != 3 || keep.size(1) != Hkv)
            value_error("keep must be [B]" + shape({Hkv}) + "[max_keep]");
        const int64_t B = keep.size(0);
        if (src.dim() != 2 || src.size(0) != B || src.size(1) == 0)
            value_error("src_table must be " + shape({B}) + "[blocks]");
        if (dst.dim() != 2 || dst.size(0) != B || dst.size(1) == 0)
            value_error("dst_table must be " + shape({B}) + "[blocks]");
        if (!sized(keep_lens, {B})) value_error("keep_lens must be " + shape({B}));
        const Place place(k_cache, "k_cache", a[6]);
        const at::ScalarType dt = k_cache.scalar_type();
        const int code = dtype_of(k_cache);
        void *kc = place(k_cache, "k_cache", dt), *vc = place(v_cache, "v_cache", dt);
        const void *sp = place(src, "src_table", at::kInt), *dp = place(dst, "dst_table", at::kInt),
                   *kp = place(keep, "keep", at::kInt), *lp = place(keep_lens, "keep_lens", at::kInt);
        const int MBs = int32_of(src.size(1), "src_table"), MBd = int32_of(dst.size(1), "dst_table"),
                  mk = int32_of(keep.size(2), "max_keep"), iB = int32_of(B, "B"),
                  iHkv = int32_of(Hkv, "Hkv"), bs = int32_of(k_cache.size(2), "block_size"),
                  d = int32_of(k_cache.size(3), "head_dim");
        launch([&] {
            return pa_compact_cache(kc, vc, static_cast<const int32_t *>(sp), MBs,
                                    static_cast<const int32_t *>(dp), MBd,
                                    static_cast<const int32_t *>(kp), mk,
                                    static_cast<const int32_t *>(lp), iB, k_cache.size(0), iHkv, bs, d,
                                    code, place.stream);
        });
        Py_RETURN_NONE;
    });
}

// q, k_cache, v_cache, block_table, context_lens, window, num_sinks, scale,
// out, stream
PyObject *decode_window(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("decode_window", 10, n, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &k_cache = tensor(a[1], "k_cache"),
                         &v_cache = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table"),
                         &lens = tensor(a[4], "context_lens");
        const int window = int32_of(a[5], "window"), sinks = int32_of(a[6], "num_sinks");
        if (q.dim() != 3 || k_cache.dim() != 4)
            value_error("q must be [B][Hq][d], pools [NB][Hkv][bs][d]");
        const int64_t B = q.size(0), d = q.size(2);
        if (k_cache.size(3) != d)
            value_error("pools must have head_dim " + std::to_string(d) + " like q");
        same_pools(k_cache, v_cache);
        if (table.dim() != 2 || table.size(0) != B)
            value_error("block_table must be " + shape({B}) + "[max_blocks_per_seq]");
        if (!sized(lens, {B})) value_error("context_lens must be " + shape({B}));
        const bool given = a[8] != Py_None;
        if (given && tensor(a[8], "out").sizes() != q.sizes())
            value_error("out must have the shape of q");
        const float scale = scale_of(a[7], d);
        const Place place(q, "q", a[9]);
        const at::ScalarType dt = k_cache.scalar_type();
        const int code = dtype_of(k_cache);
        const void *qp = place(q, "q", dt), *kc = place(k_cache, "k_cache", dt),
                   *vc = place(v_cache, "v_cache", dt), *tp = place(table, "block_table", at::kInt),
                   *lp = place(lens, "context_lens", at::kInt);
        const at::Tensor out = given ? tensor(a[8], "out") : place.new_like(q);
        void *op = place(out, "out", dt);
        const int MB = int32_of(table.size(1), "block_table"), iB = int32_of(B, "B"),
                  Hq = int32_of(q.size(1), "Hq"), Hkv = int32_of(k_cache.size(1), "Hkv"),
                  bs = int32_of(k_cache.size(2), "block_size"), id = int32_of(d, "head_dim");
        launch([&] {
            return pa_decode_window(op, qp, kc, vc, static_cast<const int32_t *>(tp), MB,
                                    static_cast<const int32_t *>(lp), iB, Hq, Hkv, id, bs,
                                    k_cache.size(0), scale, window, sinks, code, place.stream);
        });
        return THPVariable_Wrap(out);
    });
}

// q, k_cache, v_cache, block_table, query_start, context_lens, max_query_len,
// window, num_sinks, scale, out, stream
PyObject *prefill_window(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("prefill_window", 12, n, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &k_cache = tensor(a[1], "k_cache"),
                         &v_cache = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table"),
                         &start = tensor(a[4], "query_start"), &lens = tensor(a[5], "context_lens");
        const int max_query_len = int32_of(a[6], "max_query_len"), window = int32_of(a[7], "window"),
                  sinks = int32_of(a[8], "num_sinks");
        if (q.dim() != 3 || k_cache.dim() != 4 || lens.dim() != 1)
            value_error("q must be [tokens][Hq][d], pools [NB][Hkv][bs][d], context_lens [R]");
        const int64_t T = q.size(0), d = q.size(2), R = lens.size(0);
        if (k_cache.size(3) != d)
            value_error("pools must have head_dim " + std::to_string(d) + " like q");
        same_pools(k_cache, v_cache);
        if (!sized(start, {R + 1})) value_error("query_start must be " + shape({R + 1}));
        if (table.dim() != 2 || table.size(0) != R)
            value_error("block_table must be " + shape({R}) + "[max_blocks_per_seq]");
        const bool given = a[10] != Py_None;
        if (given && tensor(a[10], "out").sizes() != q.sizes())
            value_error("out must have the shape of q");
        const float scale = scale_of(a[9], d);
        const Place place(q, "q", a[11]);
        const at::ScalarType dt = k_cache.scalar_type();
        const int code = dtype_of(k_cache);
        const void *qp = place(q, "q", dt), *kc = place(k_cache, "k_cache", dt),
                   *vc = place(v_cache, "v_cache", dt), *tp = place(table, "block_table", at::kInt),
                   *sp = place(start, "query_start", at::kInt), *lp = place(lens, "context_lens", at::kInt);
        const at::Tensor out = given ? tensor(a[10], "out") : place.new_like(q);
        void *op = place(out, "out", dt);
        const int MB = int32_of(table.size(1), "block_table"), iR = int32_of(R, "R"),
                  iT = int32_of(T, "tokens"), Hq = int32_of(q.size(1), "Hq"),
                  Hkv = int32_of(k_cache.size(1), "Hkv"),
                  bs = int32_of(k_cache.size(2), "block_size"), id = int32_of(d, "head_dim");
        launch([&] {
            return pa_prefill_window(op, qp, kc, vc, static_cast<const int32_t *>(tp), MB,
                                     static_cast<const int32_t *>(sp), static_cast<const int32_t *>(lp),
                                     iR, iT, max_query_len, Hq, Hkv, id, bs, k_cache.size(0), scale,
                                     window, sinks, code, place.stream);
        });
        return THPVariable_Wrap(out);
    });
}

PyObject *set_check(PyObject *, PyObject *callable) {
    Py_INCREF(callable);
    Py_XSETREF(g_check, callable);
    Py_RETURN_NONE;
}

#define PA_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"rope_reshape_and_cache", PA_FAST(rope_reshape_and_cache)},
                          {"compact_cache", PA_FAST(compact_cache)},
                          {"decode_window", PA_FAST(decode_window)},
                          {"prefill_window", PA_FAST(prefill_window)},
                          {"set_check", set_check, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bounded_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bounded_calls() { return PyModule_Create(&kModule); }
