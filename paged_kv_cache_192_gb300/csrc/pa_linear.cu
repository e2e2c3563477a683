// Linear attention with a decay for each head, token by token:
//   S_t = l S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
// with a state S of D x D per (sequence, head), kept in 32 bits.
//
// Bound: HBM on the state (read and written once, 2 * 4 D^2 bytes per (sequence,
// head) against 8 D of q, k, v and o).  A CTA holds CW columns of one state in
// registers: a row of them is CW / 4 lanes of 16 bytes, the rows go round the
// CTA's threads, all loads of the state are issued before the first is used.
// Columns do not meet, so a state may be cut into several CTAs; o_t is a sum over
// the rows, by shuffles and then through shared memory.
//
// The same kernel takes the tokens of a request one after another, with the state
// loaded and stored once.
//
// Measured: 64 sequences of 32 heads, D 128: 42.6 us, 6.3 TB/s (0.93 of HBM); one
// sequence of 16 heads, D 64: 2.0 us on the GPU, 4.1 through the Python call; 500 tokens of
// 16 heads, D 64, fp32: 192 us, 0.38 us per token (its barrier and its sums over rows).
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "pa_linear.cuh"

namespace {

using pa::lin::LinParams;
using pa::lin::Request;

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float(float x) { return x; }
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// (Five CTAs per SM for D 64: 256 sequences of 16 heads, states in L2, 15.2 us; with four, to
// which the compiler's own choice of registers led, 17.3.)
template <typename T, int D, int CW>
__global__ void __launch_bounds__(256, D == 64 ? 5 : 4) recurrent_kernel(const LinParams p, const int32_t *added) {
    constexpr int NT = 256, LPR = CW / 4;   // lanes per row of the slice
    constexpr int RG = NT / LPR;            // rows at a time
    constexpr int NR = D / RG;              // rows per thread
    constexpr int SLICES = D / CW;
    static_assert(RG <= D && LPR <= 32, "a warp covers whole rows");
    __shared__ float sq[2][D], sk[2][D];  // the token's vectors, the next token's
    __shared__ __align__(16) float sv[2][CW];  // (read 16 bytes at a time)
    __shared__ float4 part[2][NT / 32][LPR];         // o of each warp's rows
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slice = blockIdx.x % SLICES, rh = blockIdx.x / SLICES;
    const int r = rh / p.H, h = rh % p.H;
    const int c0 = slice * CW, c = tid % LPR * 4, row0 = tid / LPR;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Request x = pa::lin::request(p, r, added);
    const T *q = static_cast<const T *>(p.q) + h * D, *k = static_cast<const T *>(p.k) + h * D,
            *v = static_cast<const T *>(p.v) + h * D + c0;
    T *out = static_cast<T *>(p.out) + static_cast<int64_t>(h) * D + c0;
    const int64_t o_stride = static_cast<int64_t>(p.H) * D;
    if (x.state < 0) {
        // padding of a batch of single tokens reads as zeros
        if (!p.query_start && tid < CW) pa::Elem<T>::store(out + r * o_stride + tid, 0.f);
        return;
    }
    float *S = p.states + (static_cast<int64_t>(x.state) * p.H + h) * (D * D) + c0 + c;
    float2 s[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const float4 x4 = x.held ? *reinterpret_cast<const float4 *>(S + (row0 + i * RG) * D) : make_float4(0.f, 0.f, 0.f, 0.f);
        s[i][0] = make_float2(x4.x, x4.y), s[i][1] = make_float2(x4.z, x4.w);
    }
    const pa::lin::Decay l = pa::lin::decay_factor(pa::lin::log_decay(p, h), 1);
    const float2 hi = make_float2(l.hi, l.hi), lo = make_float2(l.lo, l.lo);
    auto stage = [&](int t) {
        const int64_t tok = x.t0 + t;
        for (int i = tid; i < 2 * D + CW; i += NT) {
            if (i < D) sq[t & 1][i] = to_float(q[tok * p.q_stride + i]) * p.scale;
            else if (i < 2 * D) sk[t & 1][i - D] = to_float(k[tok * p.k_stride + i - D]);
            else sv[t & 1][i - 2 * D] = to_float(v[tok * p.v_stride + i - 2 * D]);
        }
    };
    stage(0);
    __syncthreads();
    for (int t = 0; t < x.n; ++t) {
        const int b = t & 1;
        if (t + 1 < x.n) stage(t + 1);
        const float4 vv = *reinterpret_cast<const float4 *>(&sv[b][c]);
        const float2 v01 = make_float2(vv.x, vv.y), v23 = make_float2(vv.z, vv.w);
        float2 o01 = make_float2(0.f, 0.f), o23 = o01;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float ki = sk[b][row0 + i * RG], qi = sq[b][row0 + i * RG];
            const float2 kk = make_float2(ki, ki), qq = make_float2(qi, qi);
            s[i][0] = pa::ffma2(hi, s[i][0], pa::ffma2(lo, s[i][0], __fmul2_rn(kk, v01)));
            s[i][1] = pa::ffma2(hi, s[i][1], pa::ffma2(lo, s[i][1], __fmul2_rn(kk, v23)));
            o01 = pa::ffma2(qq, s[i][0], o01);
            o23 = pa::ffma2(qq, s[i][1], o23);
        }
        float4 o = make_float4(o01.x, o01.y, o23.x, o23.y);
#pragma unroll
        for (int off = LPR; off < 32; off <<= 1) {
            o.x += __shfl_xor_sync(pa::kFull, o.x, off);
            o.y += __shfl_xor_sync(pa::kFull, o.y, off);
            o.z += __shfl_xor_sync(pa::kFull, o.z, off);
            o.w += __shfl_xor_sync(pa::kFull, o.w, off);
        }
        if (lane < LPR) part[b][warp][lane] = o;
        __syncthreads();  // the next token's vectors and the parts of o are there
        if (tid < CW) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < NT / 32; ++w) a += reinterpret_cast<const float *>(part[b][w])[tid];
            pa::Elem<T>::store(out + (x.t0 + t) * o_stride + tid, a);
        }
        // (part[b] and the vectors [b] are written again after the next barrier)
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
        *reinterpret_cast<float4 *>(S + (row0 + i * RG) * D) = make_float4(s[i][0].x, s[i][0].y, s[i][1].x, s[i][1].y);
}

template <typename T, int D, int CW>
int launch(const LinParams &p, const int32_t *added, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(int64_t(p.R) * p.H * (D / CW)));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    (void)cudaGetLastError();  // drop a stale error that is not ours
    const cudaError_t e = cudaLaunchKernelEx(&cfg, recurrent_kernel<T, D, CW>, p, added);
    if (e != cudaSuccess) return pa::cuda_fail(e, "linear attention launch");
    return pa::check_launch("linear attention launch");
}

// Validate mode: states in the pool and none for two requests, rows inside the
// call, lengths that hold the new tokens, decays at most 1.
int validate_linear(const LinParams &p, const int32_t *added, int max_query_len, cudaStream_t stream) try {
    std::vector<int32_t> ids(p.R), lens(p.R), qs(size_t(p.R) + 1);
    std::vector<float> decay(p.H);
    if (int rc = pa::fetch(ids.data(), p.state_ids, ids.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(lens.data(), p.context_lens, lens.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(decay.data(), p.log_decay, decay.size() * 4, stream)) return rc;
    if (const int32_t *rows = p.query_start ? p.query_start : added)
        if (int rc = pa::fetch(qs.data(), rows, qs.size() * 4, stream)) return rc;
    std::vector<bool> used(p.num_states);
    for (int r = 0; r < p.R; ++r) {
        const int64_t n = p.query_start || added ? int64_t(qs[r + 1]) - qs[r] : lens[r] != 0;
        if (n < 0 || n > max_query_len || lens[r] < n ||
            (p.query_start && n > 0 && (qs[r] < 0 || qs[r + 1] > p.T)))
            return pa::fail(PA_ERR_INVALID, "validate: request %d has %lld new tokens of %d, rows of %d, max_query_len %d",
                            r, (long long)n, lens[r], p.T, max_query_len);
        if (n == 0 || ids[r] < 0) continue;
        if (ids[r] >= p.num_states)
            return pa::fail(PA_ERR_INVALID, "validate: state_ids[%d]=%d outside the pool of %d", r, ids[r], p.num_states);
        if (used[ids[r]]) return pa::fail(PA_ERR_INVALID, "validate: state %d is named twice", ids[r]);
        used[ids[r]] = true;
    }
    for (int h = 0; h < p.H; ++h)
        if (!(decay[h] <= 0.f)) return pa::fail(PA_ERR_INVALID, "validate: log_decay[%d]=%g is positive", h, decay[h]);
    return PA_OK;
} catch (const std::bad_alloc &) {
    return pa::fail(PA_ERR_OOM, "validate: host allocation failed");
}

// The checks of both calls; PA_OK with *empty for a call without work.
int check(const char *what, const LinParams &p, int max_query_len, int D, int dtype, bool *empty) {
    *empty = false;
    if (dtype != PA_BF16 && dtype != PA_F32) return pa::fail(PA_ERR_INVALID, "%s: bad dtype", what);
    if (p.R < 0 || p.R > 65535 || p.T < 0 || p.H <= 0 || p.H > 1024 || p.num_states <= 0 || max_query_len < 0)
        return pa::fail(PA_ERR_INVALID, "%s: bad sizes", what);
    if (D != 64 && D != 128) return pa::fail(PA_ERR_UNSUPPORTED, "%s: head_dim %d unsupported", what, D);
    const int64_t row = int64_t(p.H) * D, unit = 16 / pa::dtype_size(dtype);
    for (const int64_t s : {p.q_stride, p.k_stride, p.v_stride})
        if (s < row || s % unit || s > (int64_t(1) << 28))
            return pa::fail(PA_ERR_INVALID, "%s: token stride %lld must be at least %lld, at most 2^28 and a multiple of "
                                            "16 bytes", what, (long long)s, (long long)row);
    if (!(p.scale > 0.f) || !std::isfinite(p.scale))
        return pa::fail(PA_ERR_INVALID, "%s: scale must be positive and finite", what);
    if (p.R == 0 || p.T == 0 || max_query_len == 0) {
        *empty = true;
        return PA_OK;
    }
    if (!p.out || !p.q || !p.k || !p.v || !p.states || !p.state_ids || !p.context_lens || !p.log_decay)
        return pa::fail(PA_ERR_INVALID, "%s: NULL pointer", what);
    for (const void *x : {static_cast<const void *>(p.out), p.q, p.k, p.v, static_cast<const void *>(p.states)})
        if (!pa::aligned16(x)) return pa::fail(PA_ERR_INVALID, "%s: tensors must be 16-byte aligned", what);
    return PA_OK;
}

// Whether a prompt runs on the chunk kernels: bf16 of more tokens than the recurrent
// kernel takes in the time of one chunk.  D 128: 8 tokens of 32 (request, head) pairs
// 7.3 us here and 6.9 there, of 2,048 pairs 106 and 104; 4 tokens 4.7 and 6.9, 71 and 108.
// D 64: of 32 pairs 5.1 and 5.4, but 24 tokens of 2,048 pairs 62 and 70, as an SM has room
// for many of these CTAs and one of those.
// The lengths are on the device: the call's bound and its tokens are all there is to go by.
bool uses_chunks(int R, int T, int max_query_len, int H, int D, int dtype) {
    const int most = D == 64 && int64_t(R) * H >= 4 * pa::lin::sm_count() ? 24 : 8;
    return dtype == PA_BF16 && std::min(max_query_len, T) > most;
}

size_t workspace_bytes_for(const pa::lin::Segments &s, int R, int T, int max_query_len, int H, int D, int dtype) {
    return uses_chunks(R, T, max_query_len, H, D, dtype) && s.tokens ? size_t(s.slots) * H * D * D * 4 : 0;
}

LinParams make(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
               int64_t v_stride, float *states, int num_states, const int32_t *state_ids, const int32_t *query_start,
               const int32_t *context_lens, const float *log_decay, int R, int T, int H, float scale) {
    LinParams p{};
    p.out = out;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.states = states;
    p.state_ids = state_ids;
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.log_decay = log_decay;
    p.R = R;
    p.T = T;
    p.H = H;
    p.num_states = num_states;
    p.scale = scale;
    return p;
}

}  // namespace

namespace pa {
namespace lin {

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && sms > 0)
        return sms;
    (void)cudaGetLastError();
    return 152;
}

int launch_recurrent(const LinParams &p, int D, int dtype, cudaStream_t stream, const int32_t *added) {
    // Columns per CTA: 64 (64 sequences of 32 heads, D 128: 42.4 us; 44.6 with 128, where
    // two CTAs of an SM hold too few bytes on their way between loading and storing,
    // 43.0 with 32).  A few states leave SMs idle: then 32.
    const bool cut = int64_t(p.R) * p.H < sm_count();
    auto go = [&](auto t) {
        using T = decltype(t);
        if (D == 128) return cut ? launch<T, 128, 32>(p, added, stream) : launch<T, 128, 64>(p, added, stream);
        return cut ? launch<T, 64, 32>(p, added, stream) : launch<T, 64, 64>(p, added, stream);
    };
    return dtype == PA_BF16 ? go(__nv_bfloat16()) : go(float());
}

}  // namespace lin
}  // namespace pa

extern "C" int pa_linear_decode_planned(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                        const void *v, int64_t v_stride, float *states, int num_states,
                                        const int32_t *state_ids, const int32_t *query_start,
                                        const int32_t *context_lens, const float *log_decay, int B, int H, int head_dim,
                                        float scale, int dtype, pa_stream_t stream) {
    pa::clear_error();
    LinParams p = make(out, q, q_stride, k, k_stride, v, v_stride, states, num_states, state_ids, nullptr,
                       context_lens, log_decay, B, B, H, scale);
    bool empty;
    if (int rc = check("linear_decode", p, 1, head_dim, dtype, &empty)) return rc;
    if (empty) return PA_OK;
    if (pa::validate_on())
        if (int rc = validate_linear(p, query_start, 1, stream)) return rc;
    p.err = pa::device_error_word();
    return pa::lin::launch_recurrent(p, head_dim, dtype, stream, query_start);
}

extern "C" int pa_linear_decode(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                const void *v, int64_t v_stride, float *states, int num_states,
                                const int32_t *state_ids, const int32_t *context_lens, const float *log_decay, int B,
                                int H, int head_dim, float scale, int dtype, pa_stream_t stream) {
    return pa_linear_decode_planned(out, q, q_stride, k, k_stride, v, v_stride, states, num_states, state_ids, nullptr,
                                    context_lens, log_decay, B, H, head_dim, scale, dtype, stream);
}

extern "C" int pa_linear_prefill(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                 const void *v, int64_t v_stride, float *states, int num_states,
                                 const int32_t *state_ids, const int32_t *query_start, const int32_t *context_lens,
                                 const float *log_decay, int R, int total_tokens, int max_query_len, int H,
                                 int head_dim, float scale, void *workspace, size_t workspace_bytes, int dtype,
                                 pa_stream_t stream) {
    pa::clear_error();
    LinParams p = make(out, q, q_stride, k, k_stride, v, v_stride, states, num_states, state_ids, query_start,
                       context_lens, log_decay, R, total_tokens, H, scale);
    bool empty;
    if (int rc = check("linear_prefill", p, max_query_len, head_dim, dtype, &empty)) return rc;
    if (empty) return PA_OK;
    if (!query_start) return pa::fail(PA_ERR_INVALID, "linear_prefill: NULL pointer");
    const pa::lin::Segments seg = pa::lin::segments_for(R, total_tokens, max_query_len, H);
    const size_t need = workspace_bytes_for(seg, R, total_tokens, max_query_len, H, head_dim, dtype);
    if (need && (!workspace || workspace_bytes < need))
        return pa::fail(PA_ERR_INVALID, "linear_prefill: workspace of %zu bytes, %zu needed", workspace_bytes, need);
    if (need && !pa::aligned16(workspace))
        return pa::fail(PA_ERR_INVALID, "linear_prefill: workspace must be 16-byte aligned");
    if (pa::validate_on())
        if (int rc = validate_linear(p, nullptr, max_query_len, stream)) return rc;
    p.err = pa::device_error_word();
    if (!uses_chunks(R, total_tokens, max_query_len, H, head_dim, dtype))
        return pa::lin::launch_recurrent(p, head_dim, dtype, stream);
    return pa::lin::launch_chunks(p, head_dim, max_query_len, static_cast<float *>(workspace), seg, stream);
}

extern "C" int pa_linear_prefill_workspace_size(int R, int total_tokens, int max_query_len, int H, int head_dim,
                                                int dtype, size_t *bytes) {
    pa::clear_error();
    if (!bytes) return pa::fail(PA_ERR_INVALID, "linear_prefill_workspace_size: bytes is NULL");
    if (R < 0 || R > 65535 || total_tokens < 0 || max_query_len < 0 || H <= 0 || H > 1024 ||
        (head_dim != 64 && head_dim != 128) || (dtype != PA_BF16 && dtype != PA_F32))
        return pa::fail(PA_ERR_INVALID, "linear_prefill_workspace_size: bad sizes");
    *bytes = workspace_bytes_for(pa::lin::segments_for(R, total_tokens, max_query_len, H), R, total_tokens,
                                 max_query_len, H, head_dim, dtype);
    return PA_OK;
}
