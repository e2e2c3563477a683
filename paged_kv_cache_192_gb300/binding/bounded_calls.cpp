// Torch-facing binding of the calls whose time on the host counts (rotary store,
// compaction, windowed decode and prefill; a step's plan, cross and linear attention):
// argument checks, output allocation, and the call into the C ABI of include/pa.h.
// Marshalling only, as in ops.py, whose functions forward here.
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
    // Part of `all`, from byte `at` on.
    static at::Tensor part(const at::Tensor &all, int64_t at, std::initializer_list<int64_t> dims,
                           at::ScalarType type) {
        at::Tensor t = at::detail::make_tensor<at::TensorImpl>(c10::Storage(all.storage()), all.key_set(),
                                                               c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(at / static_cast<int64_t>(c10::elementSize(type)));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(at::IntArrayRef(dims.begin(), dims.size()));
        return t;
    }
    at::Tensor new_empty(std::initializer_list<int64_t> dims, at::ScalarType type) const {
        return at::Tensor(at::detail::empty_cuda(at::IntArrayRef(dims.begin(), dims.size()), type,
                                                 c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                                 std::nullopt));
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

// seq_pages, seq_lens, free_pages, free_state, seq_ids, new_tokens, block_size,
// max_tokens, table_blocks (None: as seq_pages), out (None or five tensors),
// stream; returns the five tensors of the plan
PyObject *plan_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("plan_step", 11, n, [&]() -> PyObject * {
        const at::Tensor &pages = tensor(a[0], "seq_pages"), &lens = tensor(a[1], "seq_lens"),
                         &ring = tensor(a[2], "free_pages"), &state = tensor(a[3], "free_state"),
                         &ids = tensor(a[4], "seq_ids"), &change = tensor(a[5], "new_tokens");
        const int bs = int32_of(a[6], "block_size"), max_tokens = int32_of(a[7], "max_tokens");
        if (pages.dim() != 2 || ring.dim() != 1 || ids.dim() != 1)
            value_error("seq_pages must be [num_seqs][max_blocks], free_pages [num_blocks], seq_ids [R]");
        const int64_t S = pages.size(0), MB = pages.size(1), R = ids.size(0);
        if (!sized(lens, {S})) value_error("seq_lens must be " + shape({S}));
        if (!sized(state, {4})) value_error("free_state must be [4]");
        if (!sized(change, {R})) value_error("new_tokens must be " + shape({R}));
        if (max_tokens < 0) value_error("max_tokens must not be negative");
        int64_t W = a[8] == Py_None ? MB : int32_of(a[8], "table_blocks");
        if (W < 0) value_error("table_blocks must be positive");
        at::Tensor out[5];
        const bool given = a[9] != Py_None;
        if (given) {
            PyObject *seq = PySequence_Fast(a[9], "out must be a StepPlan");
            if (!seq) throw Raised{};
            struct Drop {
                PyObject *o;
                ~Drop() { Py_DECREF(o); }
            } drop{seq};
            if (PySequence_Fast_GET_SIZE(seq) != 5) value_error("out must be a StepPlan");
            for (int i = 0; i < 5; ++i) out[i] = tensor(PySequence_Fast_GET_ITEM(seq, i), "out");
            if (a[8] == Py_None && out[0].dim() == 2) W = out[0].size(1);
            if (!sized(out[0], {R, W}) || !sized(out[1], {R}) || !sized(out[2], {R + 1}) ||
                !sized(out[3], {max_tokens}) || !sized(out[4], {max_tokens}))
                value_error("out must be " + shape({R, W}) + ", " + shape({R}) + ", " + shape({R + 1}) + ", " +
                            shape({max_tokens}) + ", " + shape({max_tokens}));
        }
        const Place place(pages, "seq_pages", a[10]);
        void *pp = place(pages, "seq_pages", at::kInt), *lp = place(lens, "seq_lens", at::kInt),
             *rp = place(ring, "free_pages", at::kInt), *sp = place(state, "free_state", at::kInt);
        const void *ip = place(ids, "seq_ids", at::kInt), *cp = place(change, "new_tokens", at::kInt);
        if (!given) {
            // one allocation (each takes as long as the rest of the call), parts on 16 bytes
            auto whole = [](int64_t bytes) { return (bytes + 15) & ~int64_t(15); };
            const int64_t tokens = whole(8 * int64_t(max_tokens)), table = whole(4 * R * W), lens_b = whole(4 * R);
            const at::Tensor all = place.new_empty({(2 * tokens + table + lens_b + whole(4 * (R + 1))) / 8}, at::kLong);
            out[3] = Place::part(all, 0, {max_tokens}, at::kLong);
            out[4] = Place::part(all, tokens, {max_tokens}, at::kLong);
            out[0] = Place::part(all, 2 * tokens, {R, W}, at::kInt);
            out[1] = Place::part(all, 2 * tokens + table, {R}, at::kInt);
            out[2] = Place::part(all, 2 * tokens + table + lens_b, {R + 1}, at::kInt);
        }
        void *op[5];
        const char *names[5] = {"block_table", "context_lens", "query_start", "slots", "positions"};
        for (int i = 0; i < 5; ++i) op[i] = place(out[i], names[i], i < 3 ? at::kInt : at::kLong);
        const int iR = int32_of(R, "R"), iS = int32_of(S, "num_seqs"), iMB = int32_of(MB, "max_blocks"),
                  iW = int32_of(W, "table_blocks");
        launch([&] {
            return pa_plan_step(static_cast<const int32_t *>(ip), static_cast<const int32_t *>(cp), iR,
                                static_cast<int32_t *>(pp), iMB, static_cast<int32_t *>(lp), iS,
                                static_cast<int32_t *>(rp), static_cast<int32_t *>(sp), ring.size(0), bs,
                                static_cast<int32_t *>(op[0]), iW, static_cast<int32_t *>(op[1]),
                                static_cast<int32_t *>(op[2]), static_cast<int64_t *>(op[3]),
                                static_cast<int64_t *>(op[4]), max_tokens, place.stream);
        });
        PyObject *r = PyTuple_New(5);
        if (!r) throw Raised{};
        for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(r, i, THPVariable_Wrap(out[i]));
        return r;
    });
}

// q, k_cache, v_cache, block_table, query_start, encoder_lens, max_query_len,
// scale, out, stream
PyObject *cross_attention(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("cross_attention", 10, n, [&]() -> PyObject * {
        const at::Tensor &q = tensor(a[0], "q"), &k_cache = tensor(a[1], "k_cache"),
                         &v_cache = tensor(a[2], "v_cache"), &table = tensor(a[3], "block_table"),
                         &start = tensor(a[4], "query_start"), &lens = tensor(a[5], "encoder_lens");
        const int max_query_len = int32_of(a[6], "max_query_len");
        if (q.dim() != 3 || k_cache.dim() != 4 || lens.dim() != 1)
            value_error("q must be [tokens][Hq][d], pools [NB][Hkv][bs][d], encoder_lens [R]");
        const int64_t T = q.size(0), d = q.size(2), R = lens.size(0);
        if (k_cache.size(3) != d)
            value_error("pools must have head_dim " + std::to_string(d) + " like q");
        same_pools(k_cache, v_cache);
        if (!sized(start, {R + 1})) value_error("query_start must be " + shape({R + 1}));
        if (table.dim() != 2 || table.size(0) != R)
            value_error("block_table must be " + shape({R}) + "[max_blocks_per_seq]");
        const bool given = a[8] != Py_None;
        if (given && tensor(a[8], "out").sizes() != q.sizes())
            value_error("out must have the shape of q");
        const float scale = scale_of(a[7], d);
        const Place place(q, "q", a[9]);
        const at::ScalarType dt = k_cache.scalar_type();
        const int code = dtype_of(k_cache);
        const void *qp = place(q, "q", dt), *kc = place(k_cache, "k_cache", dt),
                   *vc = place(v_cache, "v_cache", dt), *tp = place(table, "block_table", at::kInt),
                   *sp = place(start, "query_start", at::kInt), *lp = place(lens, "encoder_lens", at::kInt);
        const at::Tensor out = given ? tensor(a[8], "out") : place.new_like(q);
        void *op = place(out, "out", dt);
        const int MB = int32_of(table.size(1), "block_table"), iR = int32_of(R, "R"),
                  iT = int32_of(T, "tokens"), Hq = int32_of(q.size(1), "Hq"),
                  Hkv = int32_of(k_cache.size(1), "Hkv"),
                  bs = int32_of(k_cache.size(2), "block_size"), id = int32_of(d, "head_dim");
        launch([&] {
            return pa_cross_attention(op, qp, kc, vc, static_cast<const int32_t *>(tp), MB,
                                      static_cast<const int32_t *>(sp), static_cast<const int32_t *>(lp), iR,
                                      iT, max_query_len, Hq, Hkv, id, bs, k_cache.size(0), scale, code,
                                      place.stream);
        });
        return THPVariable_Wrap(out);
    });
}

// What both linear calls take; the pointers follow once the shapes are known.
struct Linear {
    const at::Tensor &q, &k, &v, &states, &ids, &lens, &decay;
    int64_t T, H, d, R, qs, ks, vs;
    Linear(PyObject *const *a, PyObject *lens_, PyObject *decay_)
        : q(tensor(a[0], "q")), k(tensor(a[1], "k")), v(tensor(a[2], "v")), states(tensor(a[3], "states")),
          ids(tensor(a[4], "state_ids")), lens(tensor(lens_, "context_lens")), decay(tensor(decay_, "log_decay")) {
        if (q.dim() != 3 || states.dim() != 4 || ids.dim() != 1)
            value_error("q must be [tokens][H][d], states [num_states][H][d][d], state_ids [R]");
        T = q.size(0), H = q.size(1), d = q.size(2), R = ids.size(0);
        qs = token_rows(q, "q", T, H, d), ks = token_rows(k, "k", T, H, d), vs = token_rows(v, "v", T, H, d);
        if (!sized(states, {states.size(0), H, d, d}))
            value_error("states must be [num_states]" + shape({H, d, d}));
        if (!sized(lens, {R})) value_error("context_lens must be " + shape({R}));
        if (!sized(decay, {H})) value_error("log_decay must be " + shape({H}));
    }
};

// q, k, v, states, state_ids, context_lens, log_decay, scale, out, stream, query_start
// (None: every row has its token)
PyObject *linear_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("linear_decode", 11, n, [&]() -> PyObject * {
        const Linear x(a, a[5], a[6]);
        if (x.R != x.T) value_error("state_ids must be " + shape({x.T}));
        const bool planned = a[10] != Py_None;
        if (planned && !sized(tensor(a[10], "query_start"), {x.R + 1}))
            value_error("query_start must be " + shape({x.R + 1}));
        const bool given = a[8] != Py_None;
        if (given && tensor(a[8], "out").sizes() != x.q.sizes()) value_error("out must have the shape of q");
        const float scale = scale_of(a[7], x.d);
        const Place place(x.q, "q", a[9]);
        const at::ScalarType dt = x.q.scalar_type();
        const int code = dtype_of(x.q);
        const void *qp = place(x.q, "q", dt, false), *kp = place(x.k, "k", dt, false),
                   *vp = place(x.v, "v", dt, false), *ip = place(x.ids, "state_ids", at::kInt),
                   *lp = place(x.lens, "context_lens", at::kInt), *dp = place(x.decay, "log_decay", at::kFloat),
                   *tp = planned ? place(tensor(a[10], "query_start"), "query_start", at::kInt) : nullptr;
        void *sp = place(x.states, "states", at::kFloat);
        const at::Tensor out = given ? tensor(a[8], "out") : place.new_like(x.q);
        void *op = place(out, "out", dt);
        const int ns = int32_of(x.states.size(0), "num_states"), B = int32_of(x.R, "B"), H = int32_of(x.H, "H"),
                  d = int32_of(x.d, "head_dim");
        launch([&] {
            return pa_linear_decode_planned(op, qp, x.qs, kp, x.ks, vp, x.vs, static_cast<float *>(sp), ns,
                                            static_cast<const int32_t *>(ip), static_cast<const int32_t *>(tp),
                                            static_cast<const int32_t *>(lp), static_cast<const float *>(dp), B, H, d,
                                            scale, code, place.stream);
        });
        return THPVariable_Wrap(out);
    });
}

// q, k, v, states, state_ids, query_start, context_lens, max_query_len,
// log_decay, scale, out, workspace, stream
PyObject *linear_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
    return guarded("linear_prefill", 13, n, [&]() -> PyObject * {
        const Linear x(a, a[6], a[8]);
        const at::Tensor &start = tensor(a[5], "query_start");
        const int max_query_len = int32_of(a[7], "max_query_len");
        if (!sized(start, {x.R + 1})) value_error("query_start must be " + shape({x.R + 1}));
        const bool given = a[10] != Py_None;
        if (given && tensor(a[10], "out").sizes() != x.q.sizes()) value_error("out must have the shape of q");
        const float scale = scale_of(a[9], x.d);
        const Place place(x.q, "q", a[12]);
        const at::ScalarType dt = x.q.scalar_type();
        const int code = dtype_of(x.q);
        const void *qp = place(x.q, "q", dt, false), *kp = place(x.k, "k", dt, false),
                   *vp = place(x.v, "v", dt, false), *ip = place(x.ids, "state_ids", at::kInt),
                   *tp = place(start, "query_start", at::kInt), *lp = place(x.lens, "context_lens", at::kInt),
                   *dp = place(x.decay, "log_decay", at::kFloat);
        void *sp = place(x.states, "states", at::kFloat);
        const int ns = int32_of(x.states.size(0), "num_states"), R = int32_of(x.R, "R"), T = int32_of(x.T, "tokens"),
                  H = int32_of(x.H, "H"), d = int32_of(x.d, "head_dim");
        size_t bytes = 0;
        launch([&] { return pa_linear_prefill_workspace_size(R, T, max_query_len, H, d, code, &bytes); });
        at::Tensor ws;
        if (a[11] != Py_None) ws = tensor(a[11], "workspace");
        else if (bytes) ws = place.new_empty({static_cast<int64_t>((bytes + 3) / 4)}, at::kFloat);
        void *wp = ws.defined() ? place(ws, "workspace", at::kFloat) : nullptr;
        const size_t have = ws.defined() ? static_cast<size_t>(ws.numel()) * 4 : 0;
        const at::Tensor out = given ? tensor(a[10], "out") : place.new_like(x.q);
        void *op = place(out, "out", dt);
        launch([&] {
            return pa_linear_prefill(op, qp, x.qs, kp, x.ks, vp, x.vs, static_cast<float *>(sp), ns,
                                     static_cast<const int32_t *>(ip), static_cast<const int32_t *>(tp),
                                     static_cast<const int32_t *>(lp), static_cast<const float *>(dp), R, T,
                                     max_query_len, H, d, scale, wp, have, code, place.stream);
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
                          {"plan_step", PA_FAST(plan_step)},
                          {"cross_attention", PA_FAST(cross_attention)},
                          {"linear_decode", PA_FAST(linear_decode)},
                          {"linear_prefill", PA_FAST(linear_prefill)},
                          {"set_check", set_check, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_bounded_calls", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__bounded_calls() { return PyModule_Create(&kModule); }
