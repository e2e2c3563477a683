// What the translation units of linear attention share.
#pragma once

#include "pa_prefill.cuh"

namespace pa {
namespace lin {

struct LinParams {
    void *out;
    const void *q, *k, *v;  // [T][H][D], q_stride .. v_stride elements between tokens
    int64_t q_stride, k_stride, v_stride;
    float *states;  // [num_states][H][D][D]: element (i, j) belongs to k_i v_j
    const int32_t *state_ids, *query_start, *context_lens;  // query_start NULL: one token per row
    const float *log_decay;
    int *err;
    int R, T, H, num_states;
    float scale;
};

// What a request of the call is: its rows [t0, t0 + n) of q, its state, and
// whether the state holds something (else it starts from nothing).
struct Request {
    int t0, n, state;  // state -1: padding, or numbers that do not fit
    bool held;
};

__device__ __forceinline__ Request request(const LinParams &p, int r, const int32_t *added = nullptr) {
    Request x;
    const int L = p.context_lens[r];
    x.state = p.state_ids[r];
    x.t0 = p.query_start ? p.query_start[r] : r;
    x.n = p.query_start ? p.query_start[r + 1] - x.t0 : added ? added[r + 1] - added[r] : (L != 0);
    x.held = L > x.n;
    const bool padding = x.n == 0 || x.state < 0;
    if (padding || x.state >= p.num_states || x.t0 < 0 || x.n < 0 || x.n > p.T - x.t0 || L < x.n ||
        (added && x.n != 1)) {
        if (!padding) record_error(p.err, PA_DEVERR_BAD_REQUEST);
        x.state = -1;
    }
    return x;
}

// Logarithm of a head's decay.  Below -1e4 (the decay is 0 in 32 bits long before) it
// stays finite, so that l^0 is 1; a NaN stays one.
__device__ __forceinline__ float log_decay(const LinParams &p, int h) {
    const float g = p.log_decay[h];
    return g < -1e4f ? -1e4f : g;
}

// x^n = e^(g n) to within 2 ulp: g n is exact as y + rest, e^rest = 1 + rest (rest is
// below 2^-24 |y|).
__device__ __forceinline__ float decay_power(float g, int n) {
    const float y = g * n, rest = fmaf(g, static_cast<float>(n), -y), x = expf(y);
    return fmaf(x, rest, x);
}

// l^n as a sum of two numbers, so that l^n S + x is decayed(l^n, S, x): one rounding of
// the sum and one of a part that is 2^-24 of it, whatever l^n is.
//   l^n >= 1/2: hi = 1 + (l^n - 1) cut to 24 bits and what that leaves, exact: a state
//     that lives long collects no error of the factor;
//   below: hi alone (lo would add nothing to the 2 ulp of e^y; as 1 + (l^n - 1) it would
//     have an absolute error of 2^-25, all of it where l^n is small).
// lo is never 0 beside a hi that is not, so that an infinite S stays infinite.
struct Decay {
    float hi, lo;
};
__device__ __forceinline__ Decay decay_factor(float g, int n) {
    const float y = g * n;
    Decay f;
    if (y > -0.69f) {
        const float rest = fmaf(g, static_cast<float>(n), -y), e = expm1f(y), em = fmaf(rest, 1.f + e, e);
        f.hi = __fadd_rz(1.f, em);
        f.lo = em - (f.hi - 1.f);
    } else {
        f.hi = decay_power(g, n);
        f.lo = 0.f;
    }
    if (f.hi > 0.f) f.lo = fmaxf(f.lo, fmaxf(f.hi * 0x1p-60f, 0x1p-149f));
    return f;
}
__device__ __forceinline__ float decayed(const Decay &f, float s, float x) { return fmaf(f.hi, s, fmaf(f.lo, s, x)); }

// SMs of the current device; a GB300's where there is none (a workspace's size may be asked
// for anywhere).
int sm_count();

// The recurrent kernel (pa_linear.cu), any number of tokens and both types.  `added`: of a
// call without query_start, the prefix sums of the tokens that the rows gained, or NULL.
int launch_recurrent(const LinParams &p, int D, int dtype, cudaStream_t stream, const int32_t *added = nullptr);

// The kernels of long prompts (pa_linear_chunk.cu), bf16.  A call cuts its requests
// into segments of `tokens` tokens (0: it does not), at most `slots` of them, whose
// states [slots][H][D][D] fp32 are the workspace.
struct Segments {
    int tokens, slots;
};
Segments segments_for(int R, int T, int max_query_len, int H);
int launch_chunks(const LinParams &p, int D, int max_query_len, float *ws, const Segments &s, cudaStream_t stream);

}  // namespace lin
}  // namespace pa
