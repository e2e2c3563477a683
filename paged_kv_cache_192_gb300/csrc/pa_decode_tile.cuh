// Tiles of the decode kernels: one warp's attention state over staged tiles
// of one (sequence, KV head) item, on CUDA cores (WarpAttn) or on the
// warp-level tensor cores (MmaAttn), with the constants they are sized by.
#pragma once

#include "pa_device.cuh"

namespace pa {
namespace dec {

// Tuning knobs (compile-time): CTAs per SM the register budget targets, the
// per-warp staging ring, and lanes per token row for groups of <= 4 heads.
#ifndef PA_DECODE_MIN_CTAS
#define PA_DECODE_MIN_CTAS 2
#endif
#ifndef PA_DECODE_RING_KB
#define PA_DECODE_RING_KB 16
#endif
#ifndef PA_DECODE_LANES_SMALL_GROUP
#define PA_DECODE_LANES_SMALL_GROUP 8
#endif
#ifndef PA_DECODE_MIN_STEPS
#define PA_DECODE_MIN_STEPS 4  // token-row steps per tile (tile = steps x 32/G tokens)
#endif
#ifndef PA_DECODE_LOADER
#define PA_DECODE_LOADER 0  // 0: one bulk (TMA) copy per block piece; 1: per-lane cp.async
#endif
#ifndef PA_DECODE_Q_SMEM
#define PA_DECODE_Q_SMEM 0  // 1: keep the scaled q in shared memory, not registers
#endif
#ifndef PA_DECODE_MMA_MIN_GQ
#define PA_DECODE_MMA_MIN_GQ 4  // bf16 groups of at least this many heads use the tensor-core tile
#endif
#ifndef PA_DECODE_MMA_CTAS
#define PA_DECODE_MMA_CTAS 2    // CTAs per SM of the tensor-core persistent grid
#endif
constexpr int kWarps = 4;              // warps per CTA
constexpr int kMinCtas = PA_DECODE_MIN_CTAS;
constexpr int kRingBytes = PA_DECODE_RING_KB * 1024;  // per-warp K+V staging ring
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTau = 8.0f;           // lazy-rescale headroom (log2 units)

template <typename T, int D, int GQ>
struct Cfg {
    static constexpr int ES = sizeof(T);
    static constexpr int ROW = D * ES;       // bytes of one token row of one KV head
    static constexpr int CHUNKS = ROW / 16;  // 16-byte chunks per row
    static constexpr int G0 = GQ >= 8 ? 16 : PA_DECODE_LANES_SMALL_GROUP;
    static constexpr int G = G0 < CHUNKS ? G0 : CHUNKS;  // lanes per token
    static constexpr int CPL = CHUNKS / G;               // chunks per lane
    static constexpr int EPC = 16 / ES;                  // elements per chunk
    static constexpr int E = CPL * EPC;                  // elements per lane
    static constexpr int P = E / 2;                      // float2 pairs per lane
    static constexpr int TPS = 32 / G;                   // tokens per step
    static constexpr int SMIN = (G + GQ - 1) / GQ;
    static constexpr int S = SMIN > PA_DECODE_MIN_STEPS ? SMIN : PA_DECODE_MIN_STEPS;
    static constexpr int TT = S * TPS;                   // tokens per tile
    static constexpr int V = S * GQ;                     // partial dots per lane
    static constexpr int VPL = V / G;                    // scores per lane after reduction
    static constexpr int TILE = TT * ROW;                // bytes per tile per cache
    static constexpr int STAGE = 2 * TILE;               // K then V
    // stages per warp: as many as fit the ring, at least 2 when 2 fit in
    // 160 KB per CTA, else 1 (the warp then refills a stage after using it)
    static constexpr int NST = kRingBytes / STAGE >= 2 ? kRingBytes / STAGE
                               : (kWarps * 2 * STAGE <= 160 * 1024 ? 2 : 1);
    static constexpr int WARP_SMEM = NST * STAGE;
    // CTAs per SM the register budget targets (groups of 8 heads need ~220
    // registers per thread, so they run at 2)
    static constexpr int MINB = GQ >= 8 ? 2 : kMinCtas;
    static constexpr int OFF_P = kWarps * WARP_SMEM;                  // p and score buffers
    static constexpr bool QS = PA_DECODE_Q_SMEM != 0;
    static constexpr int OFF_Q = OFF_P + kWarps * 2 * TT * GQ * 4;    // scaled q (QS)
    static constexpr int OFF_BAR = OFF_Q + (QS ? kWarps * GQ * D * 4 : 0);  // mbarriers
    static constexpr int OFF_FLAG = OFF_BAR + kWarps * NST * 8;       // flag / scan scratch
    static constexpr int OFF_BT = OFF_FLAG + 16;                      // per-batch tables
    static_assert(G * CPL == CHUNKS, "row must split evenly over the lanes of a token");
    static_assert(V % G == 0 && VPL <= GQ && GQ % VPL == 0, "bad reduction shape");
    static_assert(E % 2 == 0 && TT <= 32, "bad tile");
    static_assert(GQ * D * 4 + 2 * GQ * 4 <= WARP_SMEM, "merge buffer must fit the ring");
    static_assert(kWarps * 4 <= 16, "scan scratch");
};

// Wait until the kernels this grid was launched behind (as a programmatic
// dependent) have completed and their writes are visible; a no-op for a grid
// launched without that attribute.  Every decode grid runs this before it
// reads any input.
__device__ __forceinline__ void wait_prior_grids() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Reduce V per-lane partial sums across the G lanes of a token group so that
// lane gl ends with the totals of indices [gl*V/G, (gl+1)*V/G) in v[0..V/G).
template <int V, int G>
__device__ __forceinline__ void transpose_reduce(float (&v)[V], int lane) {
#pragma unroll
    for (int m = G / 2; m >= 1; m /= 2) {
        const int half = V * m / G;
        const bool upper = (lane & m) != 0;
#pragma unroll
        for (int k = 0; k < half; ++k) {
            const float send = upper ? v[k] : v[k + half];
            const float keep = upper ? v[k + half] : v[k];
            v[k] = keep + __shfl_xor_sync(pa::kFull, send, m);
        }
    }
}

// One warp's attention state for one (sequence, KV head) item: q of the GQ
// heads (this lane's elements), running max, per-lane partial sums, and the
// PV accumulators of this lane's elements.
template <typename T, int D, int GQ>
struct WarpAttn {
    using C = Cfg<T, D, GQ>;
    int lane, gl, grp, h0, row_mine;
    float *qs;  // per-warp scaled q [GQ][D] in shared memory (QS)
    float2 q2[C::QS ? 1 : GQ][C::QS ? 1 : C::P];
    float m_run[GQ];
    float2 acc[GQ][C::P];
    float lsum[C::VPL], mh[C::VPL];
    float mhh;  // running max of head lane % GQ

    __device__ __forceinline__ void init(int lane_) {
        lane = lane_;
        gl = lane % C::G;
        grp = lane / C::G;
        // after the transpose-reduce this lane holds the scores of heads
        // h0 .. h0+VPL-1 of token row row_mine of the tile
        h0 = (gl * C::VPL) % GQ;
        row_mine = ((gl * C::VPL) / GQ) * C::TPS + grp;
    }

    // element index of pair j of chunk c of this lane
    __device__ __forceinline__ int dim_of(int c, int j) const {
        return (c * C::G + gl) * C::EPC + 2 * j;
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int h = 0; h < GQ; ++h) {
            m_run[h] = -INFINITY;
#pragma unroll
            for (int j = 0; j < C::P; ++j) acc[h][j] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < C::VPL; ++k) {
            lsum[k] = 0.f;
            mh[k] = -INFINITY;
        }
        mhh = -INFINITY;
    }

    // qb points at q[b][first head of the group][0]
    __device__ __forceinline__ void load_q(const T *qb, float qscale) {
        if constexpr (C::QS) __syncwarp();  // the previous item's reads are done
#pragma unroll
        for (int h = 0; h < GQ; ++h)
#pragma unroll
            for (int c = 0; c < C::CPL; ++c) {
                const uint4 raw =
                    *reinterpret_cast<const uint4 *>(qb + h * D + (c * C::G + gl) * C::EPC);
                float2 f[C::EPC / 2];
                pa::Elem<T>::unpack(raw, f);
#pragma unroll
                for (int i = 0; i < C::EPC / 2; ++i) {
                    const float2 v = make_float2(f[i].x * qscale, f[i].y * qscale);
                    if constexpr (C::QS) {
                        if (grp == 0)
                            *reinterpret_cast<float2 *>(qs + h * D + (c * C::G + gl) * C::EPC +
                                                        2 * i) = v;
                    } else {
                        q2[h][c * C::EPC / 2 + i] = v;
                    }
                }
            }
        if constexpr (C::QS) __syncwarp();
    }

    __device__ __forceinline__ float2 qpair(int h, int j) const {
        if constexpr (C::QS) {
            const int c = j / (C::EPC / 2), i = j % (C::EPC / 2);
            return *reinterpret_cast<const float2 *>(qs + h * D + (c * C::G + gl) * C::EPC + 2 * i);
        } else {
            return q2[h][j];
        }
    }

    // One staged tile: K rows at kaddr, V rows at vaddr (shared), nvalid rows
    // valid; with WIN, only rows [first, nvalid) are (at least one).
    template <bool WIN = false>
    __device__ __forceinline__ void tile(uint32_t kaddr, uint32_t vaddr, int nvalid, float *pbuf,
                                         float *sbuf, int first = 0) {
        const bool masked = nvalid < C::TT || (WIN && first > 0);
        // ---- QK: partial dots of S token rows x GQ heads -----------------
        float part_[C::V];
#pragma unroll
        for (int s = 0; s < C::S; ++s) {
            const int row = s * C::TPS + grp;
            float2 kf[C::P];
#pragma unroll
            for (int c = 0; c < C::CPL; ++c) {
                const uint4 raw = pa::lds128(kaddr + row * C::ROW + (c * C::G + gl) * 16);
                float2 f[C::EPC / 2];
                pa::Elem<T>::unpack(raw, f);
#pragma unroll
                for (int j = 0; j < C::EPC / 2; ++j) kf[c * C::EPC / 2 + j] = f[j];
            }
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                float2 a = make_float2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < C::P; ++j) a = pa::ffma2(qpair(h, j), kf[j], a);
                part_[s * GQ + h] = a.x + a.y;
            }
        }
        transpose_reduce<C::V, C::G>(part_, lane);

        float sc[C::VPL];
        const bool row_valid = row_mine < nvalid && (!WIN || row_mine >= first);
#pragma unroll
        for (int k = 0; k < C::VPL; ++k) sc[k] = row_valid ? part_[k] : -INFINITY;

        // ---- online softmax with lazy rescale -------------------------------
        bool need = false;
#pragma unroll
        for (int k = 0; k < C::VPL; ++k) need |= sc[k] > mh[k] + kTau;
        if (__any_sync(pa::kFull, need)) {
#pragma unroll
            for (int k = 0; k < C::VPL; ++k) sbuf[row_mine * GQ + h0 + k] = sc[k];
            __syncwarp();
            // Lane l computes head (l % GQ)'s new max and rescale factor;
            // every other value travels by shuffle (no per-lane indexing of
            // the per-head arrays, which would push them to local memory).
            const int hh = lane % GQ;
            float tmax = -INFINITY;
            for (int r = 0; r < C::TT; ++r) tmax = fmaxf(tmax, sbuf[r * GQ + hh]);
            const float mnew_l = fmaxf(mhh, tmax);
            const float alpha_l = (mhh == -INFINITY) ? 0.f : exp2f(mhh - mnew_l);
            mhh = mnew_l;
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                const float alpha = __shfl_sync(pa::kFull, alpha_l, h);
                const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
                for (int j = 0; j < C::P; ++j) acc[h][j] = __fmul2_rn(acc[h][j], a2);
                m_run[h] = __shfl_sync(pa::kFull, mnew_l, h);
            }
#pragma unroll
            for (int k = 0; k < C::VPL; ++k) {
                lsum[k] *= __shfl_sync(pa::kFull, alpha_l, h0 + k);
                mh[k] = __shfl_sync(pa::kFull, mnew_l, h0 + k);
            }
            __syncwarp();
        }
#pragma unroll
        for (int k = 0; k < C::VPL; ++k) {
            // (a head whose scores are all -inf so far takes p = 0)
            const float pk = fast_exp2(sc[k] - (WIN && mh[k] == -INFINITY ? 0.f : mh[k]));
            lsum[k] += pk;
            pbuf[row_mine * GQ + h0 + k] = pk;
        }
        __syncwarp();

        // ---- PV ---------------------------------------------------------------
#pragma unroll
        for (int s = 0; s < C::S; ++s) {
            const int row = s * C::TPS + grp;
            float prow[GQ];
            if constexpr (GQ % 4 == 0) {
#pragma unroll
                for (int h = 0; h < GQ; h += 4) {
                    const float4 t4 = *reinterpret_cast<const float4 *>(pbuf + row * GQ + h);
                    prow[h] = t4.x;
                    prow[h + 1] = t4.y;
                    prow[h + 2] = t4.z;
                    prow[h + 3] = t4.w;
                }
            } else {
#pragma unroll
                for (int h = 0; h < GQ; ++h) prow[h] = pbuf[row * GQ + h];
            }
            float2 vf[C::P];
#pragma unroll
            for (int c = 0; c < C::CPL; ++c) {
                const uint4 raw = pa::lds128(vaddr + row * C::ROW + (c * C::G + gl) * 16);
                float2 f[C::EPC / 2];
                pa::Elem<T>::unpack(raw, f);
#pragma unroll
                for (int j = 0; j < C::EPC / 2; ++j) vf[c * C::EPC / 2 + j] = f[j];
            }
            if (masked && (row >= nvalid || (WIN && row < first))) {
                // p is 0 there, but the stale row may hold NaN: 0 * NaN = NaN
#pragma unroll
                for (int j = 0; j < C::P; ++j) vf[j] = make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int h = 0; h < GQ; ++h) {
                const float2 pp = make_float2(prow[h], prow[h]);
#pragma unroll
                for (int j = 0; j < C::P; ++j) acc[h][j] = pa::ffma2(pp, vf[j], acc[h][j]);
            }
        }
    }

    // Sum acc over the token groups (every lane ends with the totals of its
    // elements) and the per-head softmax denominators over all lanes.
    __device__ __forceinline__ void reduce(float (&lh)[GQ]) {
#pragma unroll
        for (int off = C::G; off < 32; off <<= 1)
#pragma unroll
            for (int h = 0; h < GQ; ++h)
#pragma unroll
                for (int j = 0; j < C::P; ++j) {
                    acc[h][j].x += __shfl_xor_sync(pa::kFull, acc[h][j].x, off);
                    acc[h][j].y += __shfl_xor_sync(pa::kFull, acc[h][j].y, off);
                }
#pragma unroll
        for (int h = 0; h < GQ; ++h) {
            float t = 0.f;
#pragma unroll
            for (int k = 0; k < C::VPL; ++k) t += (h == h0 + k) ? lsum[k] : 0.f;
            lh[h] = t;
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1)
#pragma unroll
            for (int h = 0; h < GQ; ++h) lh[h] += __shfl_xor_sync(pa::kFull, lh[h], off);
    }

    // The whole item ended in this warp: out[h][:] = acc / lh[h] for its GQ
    // heads (outh points at the first head's row; lh from reduce()).
    __device__ __forceinline__ void store_out(T *outh, const float (&lh)[GQ]);

    // Partial of this segment: acc (unnormalised) at acc_dst + h * head_stride,
    // (max, sum) at ml_dst + h * ml_stride for each head h.
    __device__ __forceinline__ void store_partial(float *acc_dst, size_t head_stride,
                                                  float *ml_dst, size_t ml_stride,
                                                  const float (&lh)[GQ]) {
        if (grp == 0) {
#pragma unroll
            for (int h = 0; h < GQ; ++h)
#pragma unroll
                for (int cc = 0; cc < C::CPL; ++cc)
#pragma unroll
                    for (int j = 0; j < C::EPC / 2; ++j)
                        *reinterpret_cast<float2 *>(acc_dst + h * head_stride + dim_of(cc, j)) =
                            acc[h][cc * C::EPC / 2 + j];
        }
        if (lane == 0) {
#pragma unroll
            for (int h = 0; h < GQ; ++h)
                *reinterpret_cast<float2 *>(ml_dst + h * ml_stride) = make_float2(m_run[h], lh[h]);
        }
    }
};

template <typename T>
__device__ __forceinline__ void store_pair(T *dst, float a, float b);
template <>
__device__ __forceinline__ void store_pair<__nv_bfloat16>(__nv_bfloat16 *dst, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(a, b);
}
template <>
__device__ __forceinline__ void store_pair<float>(float *dst, float a, float b) {
    *reinterpret_cast<float2 *>(dst) = make_float2(a, b);
}

template <typename T, int D, int GQ>
__device__ __forceinline__ void WarpAttn<T, D, GQ>::store_out(T *outh, const float (&lh)[GQ]) {
    if (grp == 0) {
#pragma unroll
        for (int h = 0; h < GQ; ++h) {
            const float inv = 1.f / lh[h];
#pragma unroll
            for (int cc = 0; cc < C::CPL; ++cc)
#pragma unroll
                for (int j = 0; j < C::EPC / 2; ++j) {
                    const float2 a = acc[h][cc * C::EPC / 2 + j];
                    store_pair<T>(outh + h * D + dim_of(cc, j), a.x * inv, a.y * inv);
                }
        }
    }
}

// ---------------------------------------------------------------------------
// Tensor-core tile (bf16, groups of 8 heads): per 16-token tile of one
// (sequence, KV head) item, one warp computes
//   S^T[token][head] = K[token][:] . q[head][:]      (m16n8k16, M = tokens)
//   O^T[d][head]    += V^T[d][token] . P^T[token][head]   (M = head dims)
// with warp-level bf16 MMAs (fp32 accumulate).  The 8 heads of a group are
// the N = 8 columns, so no row of either product is padding.  K and V
// arrive by 2D tensor copies with the 128-byte swizzle (bank-conflict-free
// ldmatrix); q stays in registers as the B fragments of the first product,
// unscaled (S is scaled in fp32).  Lane (g, t) = (lane / 4, lane % 4) holds
// S^T for tokens g, g+8 of heads 2t, 2t+1, and O^T for dims 16m+g, 16m+g+8 of
// the same two heads, so the online softmax (max, rescale, exp, sum) needs
// no shuffle other than the per-head max over the 8 lanes of a column.  P
// enters the second product as two bf16 terms (hi + lo: p to ~2^-16
// relative), transposed into B fragments by movmatrix.  Tokens past the
// context get score -inf and their V rows are zeroed in shared memory (a
// stale row may hold NaN; 0 * NaN = NaN).
// ---------------------------------------------------------------------------
// QH: query rows carried in a stage with an item's first tile (GQ, or 2 GQ
// when an item also serves a forked child's heads in the spare columns).
template <int D, int GQ, int QH = GQ>
struct MmaCfg {
    static constexpr int TT = 16;               // tokens per tile (the M of the first product)
    static constexpr int HALVES = D / 64;       // 128-byte column blocks of a row (64 bf16)
    static constexpr int HALF = TT * 128;       // bytes of one column block of one cache's tile
    static constexpr int TILE = HALVES * HALF;  // one cache's tile
    static constexpr int QB = QH * D * 2;       // the q rows (first tile of an item)
    // K, V, then q; stages stay 1024-byte aligned for the swizzle
    static constexpr int STAGE = (2 * TILE + QB + 1023) / 1024 * 1024;
    static constexpr int NST = kRingBytes / STAGE >= 2 ? kRingBytes / STAGE : 2;
    static constexpr int WARP_SMEM = NST * STAGE;
    static constexpr int MINB = PA_DECODE_MMA_CTAS;
    static constexpr bool QS = false;
    static constexpr int OFF_P = kWarps * WARP_SMEM;  // no p / score buffers
    static constexpr int OFF_Q = OFF_P;
    static constexpr int OFF_BAR = OFF_Q;
    static constexpr int OFF_FLAG = OFF_BAR + kWarps * NST * 8;
    static constexpr int OFF_BT = OFF_FLAG + 16;
    static constexpr int KS = D / 16;           // k-steps of QK^T = m-tiles of PV
    static_assert(D % 64 == 0 && GQ <= 8 && 8 % GQ == 0 && QH <= 8, "tensor-core tile shape");
    static_assert(HALF % 1024 == 0 && STAGE % 1024 == 0, "swizzle atoms must stay aligned");
};

template <int D, int GQ, int QH = GQ>
struct MmaAttn {
    using C = MmaCfg<D, GQ, QH>;
    static constexpr int KS = C::KS;
    int lane, g, t, grp;
    float *qs;  // unused (interface of WarpAttn)
    float qscale;
    uint32_t qf[KS][2];   // B fragments of q^T: head g, dims 16k + 2t (+1) and 16k + 2t + 8 (+9)
    float acc[KS][4];     // O^T fragments: dims 16m + g (+8) x heads 2t, 2t+1
    float m_run[2], lsum[2];
    uint32_t koff[4], voff[4];  // per-lane ldmatrix row offsets (swizzled), by k-step % 4

    __device__ __forceinline__ void init(int lane_) {
        lane = lane_;
        g = lane >> 2;
        t = lane & 3;
        grp = 0;
        const int x7 = lane & 7;
        const int tk = (lane & 7) + ((lane >> 3) & 1) * 8, hk_ = lane >> 4;  // K: matrices (tok, chunk)
        const int tv = (lane & 7) + ((lane >> 4) & 1) * 8, hv = (lane >> 3) & 1;  // V^T
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            koff[j] = tk * 128 + (((2 * j + hk_) ^ x7) << 4);
            voff[j] = tv * 128 + (((2 * j + hv) ^ x7) << 4);
        }
    }

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int m = 0; m < KS; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = 0.f;
        m_run[0] = m_run[1] = -INFINITY;
        lsum[0] = lsum[1] = 0.f;
    }

    __device__ __forceinline__ void load_q(const __nv_bfloat16 *qb, float qscale_) {
        qscale = qscale_;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t b0 = 0u, b1 = 0u;
            if (g < GQ) {
                const uint32_t *row = reinterpret_cast<const uint32_t *>(qb + g * D + 16 * k);
                b0 = __ldg(row + t);
                b1 = __ldg(row + t + 4);
            }
            qf[k][0] = b0;
            qf[k][1] = b1;
        }
    }

    // q of the item from the stage (the producer copied the group's GQ rows
    // there with the item's first tile): lane (g, t) takes head g's dims
    // 16k + 2t (+1) and 16k + 2t + 8 (+9) as its B fragments.
    __device__ __forceinline__ void load_q_smem(uint32_t qaddr, float qscale_, int ncols = GQ) {
        qscale = qscale_;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t b0 = 0u, b1 = 0u;
            if (g < ncols) {
                const uint32_t a = qaddr + g * D * 2 + (16 * k + 2 * t) * 2;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b0) : "r"(a));
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b1) : "r"(a + 16));
            }
            qf[k][0] = b0;
            qf[k][1] = b1;
        }
    }

    // Column g of the products reads q row `row` (NULL: a zero column).
    __device__ __forceinline__ void load_q_row(const __nv_bfloat16 *row, float qscale_) {
        qscale = qscale_;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t b0 = 0u, b1 = 0u;
            if (row) {
                const uint32_t *r = reinterpret_cast<const uint32_t *>(row + 16 * k);
                b0 = __ldg(r + t);
                b1 = __ldg(r + t + 4);
            }
            qf[k][0] = b0;
            qf[k][1] = b1;
        }
    }

    // nvalid: tokens of the tile inside the context; with QH > GQ, the
    // columns from GQ on (a forked child's heads) see only the first
    // nvalid_hi of them.  WIN: only tokens [first, nvalid) count (at least
    // one).
    template <bool WIN = false>
    __device__ __forceinline__ void tile(uint32_t kaddr, uint32_t vaddr, int nvalid, float *,
                                         float *, int nvalid_hi = 0, int first = 0) {
        // ---- S^T = K q^T (two accumulators: shorter dependency chains) ----
        float s[4] = {0.f, 0.f, 0.f, 0.f}, s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            uint32_t a[4];
            pa::ldsm_x4(a, kaddr + (k >> 2) * C::HALF + koff[k & 3]);
            if (k & 1) pa::mma_bf16_16816(s2, a, qf[k][0], qf[k][1]);
            else pa::mma_bf16_16816(s, a, qf[k][0], qf[k][1]);
        }
        if (nvalid < C::TT) {
            // zero the V rows past the context (both column blocks)
            const int n = (C::TT - nvalid) * C::HALVES * 8;
            for (int i = lane; i < n; i += 32) {
                const int r = nvalid + i / (C::HALVES * 8), w = i % (C::HALVES * 8);
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                 vaddr + (w >> 3) * C::HALF + r * 128 + (w & 7) * 16),
                             "r"(0u)
                             : "memory");
            }
            __syncwarp();
        }
        if (WIN && first > 0) {
            // and the V rows before the first token that counts
            for (int i = lane; i < first * C::HALVES * 8; i += 32) {
                const int r = i / (C::HALVES * 8), w = i % (C::HALVES * 8);
                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                 vaddr + (w >> 3) * C::HALF + r * 128 + (w & 7) * 16),
                             "r"(0u)
                             : "memory");
            }
            __syncwarp();
        }
        const int nv = (QH > GQ && 2 * t >= GQ) ? nvalid_hi : nvalid;
        const bool v0 = g < nv && (!WIN || g >= first), v1 = g + 8 < nv && (!WIN || g + 8 >= first);
        const float x0 = v0 ? (s[0] + s2[0]) * qscale : -INFINITY;  // token g, head 2t
        const float x1 = v0 ? (s[1] + s2[1]) * qscale : -INFINITY;  // token g, head 2t+1
        const float x2 = v1 ? (s[2] + s2[2]) * qscale : -INFINITY;  // token g+8, head 2t
        const float x3 = v1 ? (s[3] + s2[3]) * qscale : -INFINITY;  // token g+8, head 2t+1
        // ---- online softmax (log2 domain, lazy rescale) ----------------------
        float mx0 = fmaxf(x0, x2), mx1 = fmaxf(x1, x3);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(pa::kFull, mx0, o));
            mx1 = fmaxf(mx1, __shfl_xor_sync(pa::kFull, mx1, o));
        }
        const bool n0 = mx0 > m_run[0] + kTau, n1 = mx1 > m_run[1] + kTau;
        if (__any_sync(pa::kFull, n0 || n1)) {
            const float m0 = n0 ? fmaxf(m_run[0], mx0) : m_run[0];
            const float m1 = n1 ? fmaxf(m_run[1], mx1) : m_run[1];
            const float a0 = m_run[0] == -INFINITY ? 0.f : exp2f(m_run[0] - m0);
            const float a1 = m_run[1] == -INFINITY ? 0.f : exp2f(m_run[1] - m1);
#pragma unroll
            for (int m = 0; m < KS; ++m) {
                acc[m][0] *= a0;
                acc[m][1] *= a1;
                acc[m][2] *= a0;
                acc[m][3] *= a1;
            }
            lsum[0] *= a0;
            lsum[1] *= a1;
            m_run[0] = m0;
            m_run[1] = m1;
        }
        // a column that has seen no token yet (m = -inf) takes p = 0, not
        // exp2(-inf + inf): the forked child's columns past its fork point
        // (WIN: columns whose scores are all -inf so far likewise)
        const float mr0 = ((QH > GQ || WIN) && m_run[0] == -INFINITY) ? 0.f : m_run[0];
        const float mr1 = ((QH > GQ || WIN) && m_run[1] == -INFINITY) ? 0.f : m_run[1];
        const float p0 = fast_exp2(x0 - mr0), p1 = fast_exp2(x1 - mr1);
        const float p2 = fast_exp2(x2 - mr0), p3 = fast_exp2(x3 - mr1);
        lsum[0] += p0 + p2;
        lsum[1] += p1 + p3;
        // ---- P^T as bf16 hi + lo B fragments --------------------------------
        const __nv_bfloat162 h01 = __floats2bfloat162_rn(p0, p1);
        const __nv_bfloat162 h23 = __floats2bfloat162_rn(p2, p3);
        const float2 f01 = __bfloat1622float2(h01), f23 = __bfloat1622float2(h23);
        const __nv_bfloat162 l01 = __floats2bfloat162_rn(p0 - f01.x, p1 - f01.y);
        const __nv_bfloat162 l23 = __floats2bfloat162_rn(p2 - f23.x, p3 - f23.y);
        const uint32_t bh0 = pa::movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h01));
        const uint32_t bh1 = pa::movmatrix_trans(*reinterpret_cast<const uint32_t *>(&h23));
        const uint32_t bl0 = pa::movmatrix_trans(*reinterpret_cast<const uint32_t *>(&l01));
        const uint32_t bl1 = pa::movmatrix_trans(*reinterpret_cast<const uint32_t *>(&l23));
        // ---- O^T += V^T P^T ---------------------------------------------------
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            uint32_t a[4];
            pa::ldsm_x4_trans(a, vaddr + (m >> 2) * C::HALF + voff[m & 3]);
            pa::mma_bf16_16816(acc[m], a, bh0, bh1);
            pa::mma_bf16_16816(acc[m], a, bl0, bl1);
        }
    }

    // Softmax sums of this lane's heads 2t, 2t+1 (reduced over the 8 lanes
    // of each column) into lh[0], lh[1].
    template <int N>
    __device__ __forceinline__ void reduce(float (&lh)[N]) const {
        static_assert(N >= 2, "two columns per lane");
        float l0 = lsum[0], l1 = lsum[1];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            l0 += __shfl_xor_sync(pa::kFull, l0, o);
            l1 += __shfl_xor_sync(pa::kFull, l1, o);
        }
        lh[0] = l0;
        lh[1] = l1;
    }

    __device__ __forceinline__ void store_out(__nv_bfloat16 *outh, const float (&lh)[GQ]) {
        static_assert(GQ % 2 == 0, "a lane's two columns are heads of one sequence");
        const float2 l = make_float2(lh[0], lh[1]);
        if (2 * t >= GQ) return;
        const float i0 = 1.f / l.x, i1 = 1.f / l.y;
        __nv_bfloat16 *o0 = outh + (2 * t) * D + g, *o1 = o0 + D;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            o0[16 * m] = __float2bfloat16_rn(acc[m][0] * i0);
            o1[16 * m] = __float2bfloat16_rn(acc[m][1] * i1);
            o0[16 * m + 8] = __float2bfloat16_rn(acc[m][2] * i0);
            o1[16 * m + 8] = __float2bfloat16_rn(acc[m][3] * i1);
        }
    }

    __device__ __forceinline__ void store_partial(float *acc_dst, size_t head_stride,
                                                  float *ml_dst, size_t ml_stride,
                                                  const float (&lh)[GQ]) {
        static_assert(GQ % 2 == 0, "a lane's two columns are heads of one sequence");
        const float2 l = make_float2(lh[0], lh[1]);
        if (2 * t >= GQ) return;
        float *a0 = acc_dst + (2 * t) * head_stride + g, *a1 = a0 + head_stride;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            a0[16 * m] = acc[m][0];
            a1[16 * m] = acc[m][1];
            a0[16 * m + 8] = acc[m][2];
            a1[16 * m + 8] = acc[m][3];
        }
        if (g == 0) {
            *reinterpret_cast<float2 *>(ml_dst + (2 * t) * ml_stride) = make_float2(m_run[0], l.x);
            *reinterpret_cast<float2 *>(ml_dst + (2 * t + 1) * ml_stride) =
                make_float2(m_run[1], l.y);
        }
    }

    // The partial of columns GQ .. 2 GQ - 1 (a forked child's heads) into the
    // child's rows: acc_dst / ml_dst address its head 0.
    __device__ __forceinline__ void store_partial_hi(float *acc_dst, size_t head_stride,
                                                     float *ml_dst, size_t ml_stride,
                                                     const float (&lh)[GQ]) {
        static_assert(QH == 2 * GQ && GQ % 2 == 0, "the child's heads fill columns GQ ..");
        const float2 l = make_float2(lh[0], lh[1]);
        const int c0 = 2 * t - GQ;
        if (c0 < 0 || c0 >= GQ) return;
        float *a0 = acc_dst + c0 * head_stride + g, *a1 = a0 + head_stride;
#pragma unroll
        for (int m = 0; m < KS; ++m) {
            a0[16 * m] = acc[m][0];
            a1[16 * m] = acc[m][1];
            a0[16 * m + 8] = acc[m][2];
            a1[16 * m + 8] = acc[m][3];
        }
        if (g == 0) {
            *reinterpret_cast<float2 *>(ml_dst + c0 * ml_stride) = make_float2(m_run[0], l.x);
            *reinterpret_cast<float2 *>(ml_dst + (c0 + 1) * ml_stride) = make_float2(m_run[1], l.y);
        }
    }
};

}  // namespace dec
}  // namespace pa
