// Rotary positions fused with the store of new K/V rows into their slots.
//
// A token's position p rotates each pair (x, y) of a query or key head by the
// angle p * f of the pair's frequency f:
//   x' = x cos - y sin,  y' = x sin + y cos
// so that q . k depends on positions by their difference only.  With several
// axes (time, height, width of an image or video patch) each frequency takes
// the position of one axis.  Values are stored as they are.
//
// Bound: memory (T * (2 Hq + 4 Hkv) rows) for long prompts, launch latency
// for decode steps.  One CTA of 128 threads per token: the token's angles are
// computed once (one thread per frequency) and used by all Hq + Hkv heads, while
// the first rows are on their way.  Measured (bf16, d 128; GPU times, calls replayed
// from a graph, a Python call takes 4 us or more): 20,001 tokens of 64/8 heads
// 122 us, 0.99 of the copy rate (137 us with 256 threads per token); 64 tokens of
// 32/8 heads 3.3 us; 2,048 tokens 11.8 us against 7.4 at that rate.  12 CTAs of 40
// registers fit an SM, 1,824 at once: 1,824 tokens take 9.5 us, 1,900 11.2, as the
// rest is a second wave with the latency of the first.  fp32: 2,048 tokens 17.9 us
// (0.83), 8,192 61.5 (0.97).  The product
// p * f and its reduction to a fraction of a turn are taken in fp64: at
// positions of 2^20 an fp32 product is off by up to 0.06 rad.
#include <cmath>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace {

constexpr int kThreads = 128;
constexpr int kMaxHalf = 256;  // frequencies (rot_dim / 2)
constexpr int kBatch = 2;      // units in flight per thread

struct RopeParams {
    uint8_t *q_out;
    const uint8_t *q, *k_new, *v_new;
    uint8_t *k_cache, *v_cache;
    const int64_t *slots, *positions;
    const float *inv_freq;
    int64_t T, num_blocks;
    int64_t q_out_stride, q_stride, k_stride, v_stride;  // bytes between tokens
    int Hq, Hkv, bs_log2, row, half;                     // row: bytes of one head
    int lanes_log2, vlanes_log2;  // lanes per rotated head, per V head (powers of two)
    int sec_end[4];                                      // first frequency past each axis
    int *err;
};

template <typename T>
__device__ __forceinline__ uint4 pack_chunk(const float2 (&f)[8 / sizeof(T)]);
template <>
__device__ __forceinline__ uint4 pack_chunk<__nv_bfloat16>(const float2 (&f)[4]) {
    uint4 r;
    uint32_t *w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[i].x, f[i].y);
        w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return r;
}
template <>
__device__ __forceinline__ uint4 pack_chunk<float>(const float2 (&f)[2]) {
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                      __float_as_uint(f[1].y));
}

__device__ __forceinline__ uint4 ld16(const uint8_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void st16(uint8_t *p, const uint4 &v) { *reinterpret_cast<uint4 *>(p) = v; }

// A unit of a rotated head is one 16-byte chunk of the first half of its
// rotated elements with the matching chunk of the second half (INTER = 0), or
// one chunk, whose pairs are adjacent (INTER = 1); chunks past the rotated
// elements are copied.  A thread requests two units at a time, the first two
// before the token's angles are computed.
template <typename T, int INTER>
__global__ void __launch_bounds__(kThreads, 12) rope_store_kernel(const RopeParams p) {
    constexpr int EPC = 16 / sizeof(T);
    constexpr int NP = EPC / 2;
    __shared__ float2 cs[kMaxHalf];
    const int64_t t = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t slot = p.slots[t];
    const int64_t blk = slot >> p.bs_log2;
    const int off = static_cast<int>(slot & ((1ll << p.bs_log2) - 1));
    const bool stored = slot >= 0 && blk < p.num_blocks;
    if (slot >= 0 && !stored && threadIdx.x == 0) pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);

    const int chunks = p.row / 16;             // per head
    const int hc = p.half / EPC;               // chunks of half the rotated elements
    const int per_head = INTER ? chunks : chunks - hc;
    const int nq = p.Hq << p.lanes_log2, nqk = nq + (p.Hkv << p.lanes_log2);
    const int total = stored ? nqk + (p.Hkv << p.vlanes_log2) : nq;
    // unit u: its source and destination rows and chunk; V chunks and chunks
    // past the rotated ones (turn = false) are copied
    struct Unit {
        const uint8_t *src;
        uint8_t *dst;
        int c;
        bool live, turn;
    };
    auto locate = [&](int u) {
        Unit x;
        const bool v = u >= nqk;
        const int lg = v ? p.vlanes_log2 : p.lanes_log2;
        const int w = v ? u - nqk : u, hh = w >> lg;
        x.c = w & ((1 << lg) - 1);
        x.live = u < total && x.c < (v ? chunks : per_head);
        x.turn = !v && x.c < (INTER ? 2 * hc : hc);
        if (!INTER && !v && !x.turn) x.c += hc;
        if (u < nq) {
            x.src = p.q + t * p.q_stride + hh * p.row;
            x.dst = p.q_out + t * p.q_out_stride + hh * p.row;
        } else {
            const int h = v ? hh : hh - p.Hq;
            const int64_t r = ((blk * p.Hkv + h) << p.bs_log2) + off;
            x.src = v ? p.v_new + t * p.v_stride + h * p.row : p.k_new + t * p.k_stride + h * p.row;
            x.dst = (v ? p.v_cache : p.k_cache) + r * p.row;
        }
        return x;
    };
    uint4 a[kBatch], b[INTER ? 1 : kBatch];
    auto request = [&](int u0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const Unit x = locate(u0 + k * kThreads);
            if (!x.live) continue;
            a[k] = ld16(x.src + x.c * 16);
            if (!INTER && x.turn) b[INTER ? 0 : k] = ld16(x.src + (x.c + hc) * 16);
        }
    };
    request(threadIdx.x);

    for (int i = threadIdx.x; i < p.half; i += kThreads) {
        const int axis = (i >= p.sec_end[0]) + (i >= p.sec_end[1]) + (i >= p.sec_end[2]);
        const double pos = static_cast<double>(p.positions[axis * p.T + t]);
        // angle in turns, reduced to [-1/2, 1/2] before it is rounded to fp32
        double turns = pos * static_cast<double>(p.inv_freq[i]) * 0.15915494309189533577;
        turns -= rint(turns);
        float s, c;
        sincospif(static_cast<float>(2.0 * turns), &s, &c);
        cs[i] = make_float2(c, s);
    }
    __syncthreads();

    for (int u0 = threadIdx.x; u0 < total; u0 += kBatch * kThreads) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const Unit x = locate(u0 + k * kThreads);
            if (!x.live) continue;
            if (!x.turn) {
                st16(x.dst + x.c * 16, a[k]);
                continue;
            }
            float2 f[NP], g[NP];
            pa::Elem<T>::unpack(a[k], f);
            if (INTER) {
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float2 w = cs[x.c * NP + i];
                    f[i] = make_float2(f[i].x * w.x - f[i].y * w.y, f[i].x * w.y + f[i].y * w.x);
                }
            } else {
                pa::Elem<T>::unpack(b[INTER ? 0 : k], g);
#pragma unroll
                for (int i = 0; i < NP; ++i) {
                    const float2 w0 = cs[x.c * EPC + 2 * i], w1 = cs[x.c * EPC + 2 * i + 1];
                    const float2 m = f[i], n = g[i];
                    f[i] = make_float2(m.x * w0.x - n.x * w0.y, m.y * w1.x - n.y * w1.y);
                    g[i] = make_float2(m.x * w0.y + n.x * w0.x, m.y * w1.y + n.y * w1.x);
                }
                st16(x.dst + (x.c + hc) * 16, pack_chunk<T>(g));
            }
            st16(x.dst + x.c * 16, pack_chunk<T>(f));
        }
        if (u0 + kBatch * kThreads < total) request(u0 + kBatch * kThreads);
    }
}

// at most 2^28 elements: a token's offset stays below 2^63 bytes
bool stride_ok(int64_t stride, int heads, int row, int es) {
    return stride > 0 && stride <= (int64_t(1) << 28) && stride * es >= int64_t(heads) * row &&
           (stride * es) % 16 == 0;
}

}  // namespace

extern "C" int pa_rope_reshape_and_cache(
    void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride, const void *k_new,
    int64_t k_stride, const void *v_new, int64_t v_stride, void *k_cache, void *v_cache,
    const int64_t *slot_mapping, const int64_t *positions, const float *inv_freq,
    const int *sections, int num_axes, int interleaved, int64_t T, int64_t num_blocks, int Hq,
    int Hkv, int block_size, int head_dim, int rot_dim, int dtype, pa_stream_t stream) {
    pa::clear_error();
    const int es = static_cast<int>(pa::dtype_size(dtype));
    if (!es) return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: bad dtype %d", dtype);
    if (T < 0 || T > INT32_MAX || num_blocks <= 0 || Hq <= 0 || Hkv <= 0 || Hq > 1024 ||
        Hkv > 1024 || head_dim <= 0 || head_dim > 1024)
        return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: bad sizes");
    if (!pa::pow2_in(block_size, 1, 1024))
        return pa::fail(PA_ERR_INVALID,
                        "rope_reshape_and_cache: block_size must be a power of two");
    if ((head_dim * es) % 16)
        return pa::fail(PA_ERR_INVALID,
                        "rope_reshape_and_cache: row bytes must be a multiple of 16");
    if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 2)
        return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: rot_dim %d must be even and at "
                                        "most head_dim", rot_dim);
    if (rot_dim / 2 > kMaxHalf || (rot_dim / 2 * es) % 16)
        return pa::fail(PA_ERR_UNSUPPORTED,
                        "rope_reshape_and_cache: rot_dim %d unsupported (half of it must be whole "
                        "16-byte chunks, at most %d elements)", rot_dim, kMaxHalf);
    if (num_axes < 1 || num_axes > 4 || !sections)
        return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: 1 to 4 axes");
    RopeParams p{};
    int64_t end = 0;
    for (int a = 0; a < 4; ++a) {
        if (a < num_axes) {
            if (sections[a] < 0) return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: negative section");
            end += sections[a];
        }
        p.sec_end[a] = static_cast<int>(end < rot_dim ? end : rot_dim);
    }
    if (end != rot_dim / 2)
        return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: sections sum to %lld, not to "
                                        "rot_dim / 2 = %d", (long long)end, rot_dim / 2);
    const int row = head_dim * es;
    if (!stride_ok(q_stride, Hq, row, es) || !stride_ok(q_out_stride, Hq, row, es) ||
        !stride_ok(k_stride, Hkv, row, es) || !stride_ok(v_stride, Hkv, row, es))
        return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: a token stride is shorter than "
                                        "its heads, above 2^28 or no multiple of 16 bytes");
    if (T == 0) return PA_OK;
    if (!q_out || !q || !k_new || !v_new || !k_cache || !v_cache || !slot_mapping || !positions ||
        !inv_freq)
        return pa::fail(PA_ERR_INVALID, "rope_reshape_and_cache: NULL pointer");
    for (const void *x : {static_cast<const void *>(q_out), q, k_new, v_new,
                          static_cast<const void *>(k_cache), static_cast<const void *>(v_cache)})
        if (!pa::aligned16(x))
            return pa::fail(PA_ERR_INVALID,
                            "rope_reshape_and_cache: pointers must be 16-byte aligned");
    if (pa::validate_on())
        if (int rc = pa::validate_slots(slot_mapping, T, num_blocks, block_size, stream)) return rc;
    p.q_out = static_cast<uint8_t *>(q_out);
    p.q = static_cast<const uint8_t *>(q);
    p.k_new = static_cast<const uint8_t *>(k_new);
    p.v_new = static_cast<const uint8_t *>(v_new);
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.slots = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.T = T;
    p.num_blocks = num_blocks;
    p.q_out_stride = q_out_stride * es;
    p.q_stride = q_stride * es;
    p.k_stride = k_stride * es;
    p.v_stride = v_stride * es;
    p.Hq = Hq;
    p.Hkv = Hkv;
    while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
    p.row = row;
    p.half = rot_dim / 2;
    const int chunks = row / 16, per_head = interleaved ? chunks : chunks - p.half * es / 16;
    while ((1 << p.lanes_log2) < per_head) ++p.lanes_log2;
    while ((1 << p.vlanes_log2) < chunks) ++p.vlanes_log2;
    p.err = pa::device_error_word();
    (void)cudaGetLastError();  // drop a stale error that is not ours
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(T));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (dtype == PA_BF16)
        e = interleaved ? cudaLaunchKernelEx(&cfg, rope_store_kernel<__nv_bfloat16, 1>, p)
                        : cudaLaunchKernelEx(&cfg, rope_store_kernel<__nv_bfloat16, 0>, p);
    else
        e = interleaved ? cudaLaunchKernelEx(&cfg, rope_store_kernel<float, 1>, p)
                        : cudaLaunchKernelEx(&cfg, rope_store_kernel<float, 0>, p);
    if (e != cudaSuccess) return pa::cuda_fail(e, "rope_reshape_and_cache launch");
    return pa::check_launch("rope_reshape_and_cache launch");
}
