// Chunked prefill with a sliding window and sinks over a paged KV cache
// (bf16, tcgen05).
//
// New token i of request r sits at position p = P_r + i and sees
//   j <= p  with  j < S (sinks)  or  j > p - W (the window, itself included).
// Blocks of the table that no query of the chunk sees are never read: their
// pages may have been freed and their entries may be anything.
//
// Bound: tensor cores (4 D flop per visible (query, key) pair and head, half
// as much again for the second term of P).  The machinery is that of the
// persistent prefill kernel (one CTA per SM running a list of work items
// through warp-specialised pipelines); what differs is what an item reads.
// A work item is (request, 256 query rows, KV head); its keys are the sink
// tiles and the tiles from the window of its first query to its last query's
// own position, so its cost does not grow with the context.  The list of all
// items follows from the requests' lengths (a prefix sum in shared memory,
// the same in every CTA): CTA c takes items c, c + gridDim.x, ...  K/V tiles
// of 64 tokens arrive by TMA, through table entries that the loader warp
// fetches 32 at a time, one batch ahead, so a table may have any length.
//
// Warps: 0-3 and 4-7 softmax of groups A and B; 8 and 11 issue the
// tcgen05.mma of A and of B; 9 loads K/V; 10 loads the query tiles.  TMEM (512
// columns): O_A [0,128), O_B [128,256), then per group 64 columns of S and 64
// of P (bf16 hi, lo: ~2^-16 of a weight).  Every wait is bounded.
//
// That kernel's groups are an item's two query tiles of 128 rows, and both use
// every K/V tile.  Batches of so few items that SMs would stay idle run on
// prefill_window_split_kernel instead: an item is one query tile, a cluster of
// up to 8 CTAs divides its K/V tiles, and within a CTA group A takes the even
// tiles and B the odd ones; the partial results meet through distributed shared
// memory by log-sum-exp.
//
// Measured (32/8 heads, d 128): a prompt of 16,384 tokens with window 4096 and 64
// sinks 868 to 901 us, 1,080 to 1,120 TFLOP/s (0.64 to 0.66 of cuBLAS's sustained
// bf16).  A 64-key tile
// of both groups takes 1,870 cycles, of which the tensor core needs 1,790: PV
// twice 512 for the two terms of P, and S twice 384 instead of 256, as it reads
// 192 bytes of shared memory per cycle of its own (128-row A and 64-row B against
// 64 columns).  4 chunks of 512 tokens over up to 3,584 earlier ones, window
// 1024: 47 us: 256 items of 1 to 19 tiles on 152 SMs, 37 tiles on the fullest, 25 on
// average.  One chunk of 40 tokens, window 513: 9.9 us.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "pa_prefill.cuh"

namespace {

using namespace pa::pf;

constexpr int kMaxR = 256;  // requests per launch (the tables in shared memory)

struct WinParams {
    __nv_bfloat16 *out;
    const int32_t *block_table, *query_start, *context_lens;
    int *err;
    int64_t num_blocks;
    int R, T, Hq, Hkv, bs, bs_log2, MB, window, sinks;
    float qscale;  // scale * log2(e)
};

// Tables of the requests, shared by both kernels' layouts.
struct ReqTables {
    int pre[kMaxR + 1];  // query tiles before request r
    int qs[kMaxR], n[kMaxR], L[kMaxR];
    int scan[12];
};

template <int D>
struct WLayout {
    static constexpr int NST = 4;
    static constexpr int THREADS = 12 * 32;
    static constexpr int MMA_WARP = 8, LOAD_WARP = 9, Q_WARP = 10, MMA_WARP_B = 11;
    static constexpr int TMEM_COLS = 512;
    static constexpr int QT_BYTES = 128 * D * 2;   // one query tile
    static constexpr int T_BYTES = kT2KT * D * 2;  // one K or V tile
    static constexpr int OFF_KV = 2 * QT_BYTES;    // [stage][K|V]
    static constexpr int OFF_BAR = OFF_KV + NST * 2 * T_BYTES;
    // kv_full, kv_empty [NST]; s_full, s_free, p_full, o_done, o_free [2];
    // q_full, q_empty, drain
    static constexpr int N_BAR = 2 * NST + 10 + 3;
    static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;  // TMEM slot, fail flag
    static constexpr int OFF_REQ = OFF_MISC + 16;
    static constexpr int OFF_OUT = (OFF_REQ + int(sizeof(ReqTables)) + 15) / 16 * 16;  // 2 KB per warp
    static constexpr int SMEM = OFF_OUT + 8 * 2048 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(OFF_BAR % 8 == 0 && OFF_REQ % 4 == 0, "alignment");
};

// The split kernel: one query tile, and rings of their own for K and V (a K
// tile is free once its scores are there, a V tile only after the softmax).
// At the end the rings' place holds what the cluster's CTAs send of this CTA's
// columns, [C][D / C / 4][128] x 4 columns, and behind it what the two groups
// exchange, [2][D / 8][128] x 4; the query tile's place holds the (max, sum) of
// each, [C][128] and [2][128].
template <int D>
struct SLayout {
    static constexpr int NST = 5;
    static constexpr int THREADS = 12 * 32;
    static constexpr int MMA_WARP = 8, K_WARP = 9, V_WARP = 10, MMA_WARP_B = 11;
    static constexpr int TMEM_COLS = 512;
    static constexpr int QT_BYTES = 128 * D * 2;
    static constexpr int T_BYTES = kT2KT * D * 2;
    static constexpr int MAX_C = D / 16;  // a CTA finishes at least 16 columns
    static constexpr int OFF_K = QT_BYTES;
    static constexpr int OFF_V = OFF_K + NST * T_BYTES;
    static constexpr int OFF_BAR = OFF_V + NST * T_BYTES;
    // k_full, k_empty, v_full, v_empty [NST]; s_full, s_free, p_full, o_done [2];
    // q_full, drain
    static constexpr int N_BAR = 4 * NST + 8 + 2;
    static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;
    static constexpr int OFF_REQ = OFF_MISC + 16;
    static constexpr int SMEM = OFF_REQ + int(sizeof(ReqTables)) + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static constexpr int X_BYTES = 128 * D * 4;  // received, and as much exchanged
    static_assert(2 * X_BYTES <= OFF_BAR - OFF_K, "the partial O must fit the rings");
    static_assert((MAX_C + 2) * 128 * 8 <= QT_BYTES, "(max, sum) must fit the query tile");
    static_assert(OFF_BAR % 8 == 0 && OFF_REQ % 4 == 0, "alignment");
};

// Query rows t0 .. of request r (its tokens are rows qs.. of q, n new ones at
// positions P..), KV head hk; keys [0, kv_end) of which [S, lo) are hidden
// from every row.  Tiles 0..ns-1 start at token 0, the others at wbase.
struct Item {
    int r, qs, n, P, t0, hk, kv_end, lo, ns, wbase, ntiles;
    __device__ __forceinline__ int base(int j) const {
        return j < ns ? j * kT2KT : wbase + (j - ns) * kT2KT;
    }
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(pa::smem_u32(bar))
        : "memory");
}

// The requests of a launch and the prefix sum of their query tiles of `qtok`
// tokens into the tables; returns the number of tiles.  A request whose numbers
// do not fit gets none.  Whole CTA of 12 warps; ends with a barrier.
__device__ __forceinline__ int read_requests(const WinParams &p, ReqTables &t, int qtok) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int carry = 0;
    for (int r0 = 0; r0 < p.R; r0 += 12 * 32) {
        const int r = r0 + tid;
        int np = 0;
        if (r < p.R) {
            const int qs = p.query_start[r], n = p.query_start[r + 1] - qs, L = p.context_lens[r];
            if (n > 0 && qs >= 0 && n <= p.T - qs && L >= n && L <= p.MB << p.bs_log2)
                np = (n + qtok - 1) / qtok;
            else if (n != 0 || L < 0 || L > p.MB << p.bs_log2)
                pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
            t.qs[r] = qs;
            t.n[r] = n;
            t.L[r] = L;
        }
        int x = np;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(pa::kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) t.scan[warp] = x;
        __syncthreads();
        int off = carry;
        for (int w = 0; w < 12; ++w) {
            off += w < warp ? t.scan[w] : 0;
            carry += t.scan[w];
        }
        if (r < p.R) t.pre[r + 1] = off + x;
        __syncthreads();
    }
    if (tid == 0) t.pre[0] = 0;
    __syncthreads();
    return carry;
}

__device__ __forceinline__ Item make_item(const WinParams &p, const ReqTables &t, int x, int qtok) {
    Item it;
    const int pair = x / p.Hkv;
    it.hk = x % p.Hkv;
    int lo = 0, hi = p.R - 1;  // the last request with pre[r] <= pair
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.pre[mid] <= pair) lo = mid;
        else hi = mid - 1;
    }
    it.r = lo;
    // the last query tiles first: they see the most keys
    it.t0 = (t.pre[lo + 1] - 1 - pair) * qtok;
    it.qs = t.qs[lo];
    it.n = t.n[lo];
    it.P = t.L[lo] - it.n;
    it.kv_end = min(it.P + it.n, it.P + it.t0 + qtok);
    it.lo = max(0, it.P + it.t0 - p.window + 1);
    it.ns = (min(p.sinks, it.kv_end) + kT2KT - 1) / kT2KT;
    const int w0 = it.lo / kT2KT, w1 = (it.kv_end + kT2KT - 1) / kT2KT;
    if (w0 <= it.ns) {  // the window reaches the sinks' tiles: one range
        it.ns = 0;
        it.wbase = 0;
        it.ntiles = w1;
    } else {
        it.wbase = w0 * kT2KT;
        it.ntiles = it.ns + w1 - w0;
    }
    return it;
}

// Pool rows of an item's (tile, block) slots, 32 at a time, one per lane, the
// next batch fetched one batch ahead; tiles j0, j0 + 1, ... in order.  A block
// that no row of the item sees is out of bounds: zero-filled, not read.
struct RowFetch {
    const WinParams &p;
    const Item &I;
    const int32_t *bt;
    int lane, end, nb, tpb, rows_total, tb, row, row_next;
    __device__ __forceinline__ RowFetch(const WinParams &p_, const Item &I_, int lane_, int j0, int end_)
        : p(p_), I(I_), lane(lane_), end(end_) {
        bt = p.block_table + static_cast<size_t>(I.r) * p.MB;
        nb = max(1, kT2KT >> p.bs_log2);  // blocks per tile
        tpb = 32 / nb;                    // tiles per batch
        rows_total = static_cast<int>(p.num_blocks * p.Hkv) << p.bs_log2;
        tb = j0;
        row = fetch(j0);
        row_next = fetch(j0 + tpb);
    }
    __device__ __forceinline__ int fetch(int t) const {
        const int j = t + lane / nb;
        if (j >= end) return rows_total;
        const int tok = I.base(j) + (lane % nb) * p.bs;
        const int blk0 = tok & ~(p.bs - 1);  // (blocks of 128: the tile is half of one)
        if (tok >= I.kv_end || (tok >= p.sinks && blk0 + p.bs <= I.lo)) return rows_total;
        int v = __ldg(bt + (tok >> p.bs_log2));
        if (v < 0 || v >= p.num_blocks) {
            pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
            v = 0;
        }
        return ((v * p.Hkv + I.hk) << p.bs_log2) + (tok & (p.bs - 1));
    }
    // Slots of tile j; lane slot0 + k then holds the row of its k-th block.
    __device__ __forceinline__ int advance(int j) {
        if (j - tb >= tpb) {
            tb += tpb;
            row = row_next;
            row_next = fetch(tb + tpb);
        }
        return (j - tb) * nb;
    }
};

// One 64-key tile of one row (this thread's): scores from TMEM, which is then
// released, hidden keys masked, and the weights as two bf16 terms (hi + lo).
// Hidden are the keys past hi and keys [s0, wl] (relative to the tile).
// Returns the factor by which the row's earlier sums shrink.
__device__ __forceinline__ float softmax_tile(uint32_t s_addr, uint64_t *s_free, int lane, int hi,
                                              int wl, int s0, float qs2, float &m_used, float &lsum,
                                              uint32_t (&ph)[32], uint32_t (&pl)[32]) {
    uint32_t sr[2][32];
    pa::tc::ld32(s_addr, sr[0]);
    pa::tc::ld32(s_addr + 32, sr[1]);
    pa::tc::wait_ld();
    // S may now be overwritten by the next tile's
    pa::tc::fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(s_free);
    float s[64];
#pragma unroll
    for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(sr[c >> 5][c & 31]);
    if (hi < kT2KT - 1 || (wl >= 0 && s0 < kT2KT)) {
        // bit c: key c of the tile is hidden; up(n): the bits from n on
        auto up = [](int n) { return n >= 64 ? 0ull : ~0ull << max(n, 0); };
        const uint64_t hidden = up(hi + 1) | (up(s0) & ~up(wl + 1));
        const uint32_t hl = static_cast<uint32_t>(hidden), hh = static_cast<uint32_t>(hidden >> 32);
#pragma unroll
        for (int c = 0; c < 64; ++c)
            if ((c < 32 ? hl : hh) & (1u << (c & 31))) s[c] = -INFINITY;
    }
    float mx[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float m3 = max3f(s[e], s[8 + e], s[16 + e]);
        m3 = max3f(m3, s[24 + e], s[32 + e]);
        m3 = max3f(m3, s[40 + e], s[48 + e]);
        mx[e] = fmaxf(m3, s[56 + e]);
    }
    const float tmax = max3f(max3f(mx[0], mx[1], mx[2]), max3f(mx[3], mx[4], mx[5]),
                             fmaxf(mx[6], mx[7])) *
                       qs2;
    float alpha = 1.f;
    if (tmax > m_used + kTcTau) {
        alpha = (m_used == -INFINITY) ? 0.f : exp2f(m_used - tmax);
        m_used = tmax;
    }
    float2 rs2[4] = {};
    // (a row that has seen no key yet takes p = 0, not exp2(-inf + inf))
    const float mr = m_used == -INFINITY ? 0.f : m_used;
    const float2 q2 = make_float2(qs2, qs2), nm2 = make_float2(-mr, -mr);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        const float2 e = pa::ffma2(make_float2(s[2 * c], s[2 * c + 1]), q2, nm2);
        const float p0 = fast_exp2(e.x);
        const float p1 = fast_exp2(e.y);
        rs2[c & 3] = __fadd2_rn(rs2[c & 3], make_float2(p0, p1));
        ph[c] = pack_bf16(p0, p1);
        const float2 lo = pa::ffma2(pa::bf16x2_to_float2(ph[c]), make_float2(-1.f, -1.f),
                                    make_float2(p0, p1));
        pl[c] = pack_bf16(lo.x, lo.y);
    }
    const float rs = ((rs2[0].x + rs2[0].y) + (rs2[1].x + rs2[1].y)) +
                     ((rs2[2].x + rs2[2].y) + (rs2[3].x + rs2[3].y));
    lsum = lsum * alpha + rs;
    return alpha;
}

// O of this thread's row times alpha (its products so far are complete).
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t o_addr, float alpha) {
    if (!__any_sync(pa::kFull, alpha != 1.f)) return;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t o[32];
        pa::tc::ld32(o_addr + c0, o);
        pa::tc::wait_ld();
#pragma unroll
        for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
        pa::tc::st32(o_addr + c0, o);
    }
}

// V rows of a tile that no row of the item sees may hold anything (slots never
// written, tokens before the window): P is 0 there, but 0 * NaN is NaN, so
// they are zeroed before P arrives.  j0: the tile's first token.
__device__ __forceinline__ bool has_hidden_rows(const Item &I, int sinks, int j0) {
    return I.kv_end - j0 < kT2KT || max(0, sinks - j0) < min(kT2KT, I.lo - j0);
}
template <int D>
__device__ __forceinline__ void zero_hidden_rows(const Item &I, int sinks, int j0, uint32_t vst,
                                                 int row) {
    constexpr int CH = D * 2 / 16;  // 16-byte chunks per row
    auto zero = [&](int a, int b) {
        for (int idx = row; idx < (b - a) * CH; idx += 128)
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                             vst + pa::tc::sw128(a + idx / CH, idx % CH * 8, kT2KT)),
                         "r"(0u)
                         : "memory");
    };
    zero(min(I.kv_end - j0, kT2KT), kT2KT);
    const int ha = max(0, sinks - j0), hb = min(kT2KT, I.lo - j0);
    if (ha < hb) zero(ha, hb);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// P of this thread's row (hi, then lo) into TMEM.
__device__ __forceinline__ void put_p(uint32_t p_addr, const uint32_t (&ph)[32],
                                      const uint32_t (&pl)[32]) {
    pa::tc::st32(p_addr, ph);
    pa::tc::st32(p_addr + 32, pl);
    pa::tc::wait_st();
    pa::tc::fence_before();
    __syncwarp();
}

// S (TMEM) = Q tile x K tile^T
template <int D>
__device__ __forceinline__ void mma_s(uint32_t s_col, uint64_t dq, uint64_t dk) {
    constexpr uint32_t kIdS = pa::tc::idesc_bf16(128, kT2KT, 0, 0);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
        pa::tc::mma_ss(s_col, dq + (((ks >> 2) * 128 * 128 + (ks & 3) * 32) >> 4),
                       dk + (((ks >> 2) * kT2KT * 128 + (ks & 3) * 32) >> 4), kIdS, ks > 0);
}

// O (+)= P_hi V + P_lo V
template <int D>
__device__ __forceinline__ void mma_pv(uint32_t o_col, uint32_t p_col, uint64_t dv, int accumulate) {
    constexpr uint32_t kIdO = pa::tc::idesc_bf16(128, D, 0, 1);
#pragma unroll
    for (int ks = 0; ks < kT2KT / 16; ++ks) {
        const uint64_t b = dv + ((ks * 16 * 128) >> 4);
        pa::tc::mma_ts(o_col, p_col + ks * 8, b, kIdO, ks == 0 ? accumulate : 1);
        pa::tc::mma_ts(o_col, p_col + 32 + ks * 8, b, kIdO, 1);
    }
}

__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity) {
    return __all_sync(pa::kFull, pa::mbar_wait(bar, parity));
}

template <int D, int GQ>
__global__ void __launch_bounds__(WLayout<D>::THREADS, 1)
    prefill_window_kernel(const WinParams p, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap qmap) {
    using Lay = WLayout<D>;
    constexpr int NST = Lay::NST;
    constexpr int QTOK = 256 / GQ;  // query tokens per item
    constexpr int TILE_TX = 2 * Lay::T_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sq = pa::smem_u32(smem), skv = sq + Lay::OFF_KV;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *kv_full = bars, *kv_empty = bars + NST;
    uint64_t *s_full = bars + 2 * NST, *s_free = s_full + 2;  // [group]
    uint64_t *p_full = s_free + 2, *o_done = p_full + 2, *o_free = o_done + 2;
    uint64_t *q_full = o_free + 2, *q_empty = q_full + 1, *drain = q_empty + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_MISC);
    volatile int *fail = reinterpret_cast<volatile int *>(smem + Lay::OFF_MISC + 4);
    ReqTables &req = *reinterpret_cast<ReqTables *>(smem + Lay::OFF_REQ);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // ---- set-up: barriers, TMEM ------------------------------------------------
    if (tid == 0) {
        for (const CUtensorMap *map : {&kmap, &vmap, &qmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
        for (int i = 0; i < NST; ++i) {
            pa::mbar_init(&kv_full[i], 1);
            pa::mbar_init(&kv_empty[i], 2);  // both groups' PV
        }
        for (int i = 0; i < 2; ++i) {
            pa::mbar_init(&s_full[i], 1);
            pa::mbar_init(&s_free[i], 4);  // one arrival per softmax warp
            pa::mbar_init(&p_full[i], 4);
            pa::mbar_init(&o_done[i], 1);
            pa::mbar_init(&o_free[i], 4);
        }
        pa::mbar_init(q_full, 1);
        pa::mbar_init(q_empty, 2);  // both groups' last S
        pa::mbar_init(drain, 2);
        *fail = 0;
        pa::fence_barrier_init();
    }
    if (warp == Lay::MMA_WARP) pa::tc::alloc(tslot, Lay::TMEM_COLS);
    pa::tc::fence_before();
    __syncthreads();
    pa::tc::fence_after();
    const uint32_t tmem = *tslot;
    // launched as a programmatic dependent: the inputs are ready past this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int nitems = read_requests(p, req, QTOK) * p.Hkv;
    auto item_of = [&](int x) { return make_item(p, req, x, QTOK); };

    int loads_issued = 0;  // loader lane 0: K/V tiles issued (for the drain after a failure)

    if (warp == Lay::Q_WARP) {
        // ---------------- query tiles ----------------
        // Rows m = 128 * tile + i: query token t0 + m / GQ, head hk * GQ + m % GQ.
        // Whole tiles are copied: rows past the request's new tokens are another
        // request's (or zeros past the last), are never stored, and as a row's
        // scores and output depend on that row alone they affect nothing.
        int it = 0;
        for (int x = blockIdx.x; x < nitems && !*fail; x += gridDim.x, ++it) {
            const Item I = item_of(x);
            if (it > 0 && !wait_all(q_empty, (it - 1) & 1)) {
                *fail = 1;
                break;
            }
            if (lane == 0) {
                pa::mbar_arrive_expect_tx(q_full, 2 * Lay::QT_BYTES);
                for (int qt = 0; qt < 2; ++qt)
#pragma unroll
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_3d(sq + qt * Lay::QT_BYTES + h * (128 * 128), &qmap, h * 64,
                                    I.hk * GQ, I.qs + I.t0 + qt * (128 / GQ), q_full);
            }
            __syncwarp();
        }
        // the last copies must have landed before the CTA may exit
        if (it > 0) (void)pa::mbar_wait(q_full, (it - 1) & 1);
    } else if (warp == Lay::LOAD_WARP) {
        // ---------------- K/V loader ----------------
        int g = 0;  // CTA-wide K/V tile counter
        for (int x = blockIdx.x; x < nitems && !*fail; x += gridDim.x) {
            const Item I = item_of(x);
            RowFetch rf(p, I, lane, 0, I.ntiles);
            bool ok = true;
            for (int j = 0; j < I.ntiles && ok; ++j, ++g) {
                const int st = g % NST, slot0 = rf.advance(j);
                if (g >= NST) ok = wait_all(&kv_empty[st], ((g / NST) - 1) & 1);
                if (!ok) break;
                const uint32_t kst = skv + st * 2 * Lay::T_BYTES, vst = kst + Lay::T_BYTES;
                if (lane == 0) {
                    pa::mbar_arrive_expect_tx(&kv_full[st], TILE_TX);
                    ++loads_issued;
                }
                __syncwarp();
                // the lane that holds a block's row issues its copies
                if (lane >= slot0 && lane < slot0 + rf.nb) {
                    const uint32_t b = static_cast<uint32_t>(lane - slot0) * p.bs * 128;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        const uint32_t off = h * kT2KT * 128 + b;
                        tma_load_2d(kst + off, &kmap, h * 64, rf.row, &kv_full[st]);
                        tma_load_2d(vst + off, &vmap, h * 64, rf.row, &kv_full[st]);
                    }
                }
                __syncwarp();
            }
            if (!ok) *fail = 1;
        }
    } else if (warp == Lay::MMA_WARP || warp == Lay::MMA_WARP_B) {
        // ---------------- MMA issuers, one per group ----------------
        const int wg = warp == Lay::MMA_WARP ? 0 : 1;
        constexpr uint32_t kStage = (2 * Lay::T_BYTES) >> 4;
        const uint64_t dq = pa::tc::sdesc(sq, 16, 1024) +
                            static_cast<uint32_t>(wg * (Lay::QT_BYTES >> 4));
        const uint64_t dk = pa::tc::sdesc(skv, 16, 1024);
        const uint64_t dv = pa::tc::sdesc(skv + Lay::T_BYTES, kT2KT * 128, 1024);
        const uint32_t sc = tmem + 256 + wg * 128, od = tmem + wg * 128;
        // S of CTA tile g once its K has landed and the group has loaded the
        // S before it
        auto start = [&](int g) {
            if (!wait_all(&kv_full[g % NST], (g / NST) & 1)) return false;
            if (g > 0 && !wait_all(&s_free[wg], (g - 1) & 1)) return false;
            pa::tc::fence_after();
            if (pa::tc::elect_one()) {
                mma_s<D>(sc, dq, dk + static_cast<uint32_t>((g % NST) * kStage));
                pa::tc::commit(&s_full[wg]);
            }
            __syncwarp();
            return true;
        };
        bool ok = true;
        int g = 0, it = 0;
        for (int x = blockIdx.x; ok && x < nitems; x += gridDim.x, ++it) {
            const int nt = item_of(x).ntiles;
            ok = wait_all(q_full, it & 1) && start(g);
            for (int j = 0; j < nt && ok; ++j, ++g) {
                if (j + 1 < nt) {
                    ok = start(g + 1);
                    if (!ok) break;
                } else {
                    if (pa::tc::elect_one()) pa::tc::commit(q_empty);
                    __syncwarp();
                }
                // the item's first PV overwrites O once the group has read the last item's
                if (j == 0 && it > 0) ok = wait_all(&o_free[wg], (it - 1) & 1);
                if (ok) ok = wait_all(&p_full[wg], g & 1);
                if (!ok) break;
                pa::tc::fence_after();
                if (pa::tc::elect_one()) {
                    mma_pv<D>(od, sc + 64, dv + static_cast<uint32_t>((g % NST) * kStage), j > 0);
                    pa::tc::commit(&o_done[wg]);
                    pa::tc::commit(&kv_empty[g % NST]);
                }
                __syncwarp();
            }
        }
        if (!ok) *fail = 1;
    } else {
        // ---------------- softmax warp groups ----------------
        const int wg = warp >> 2;   // query tile A or B
        const int row = tid & 127;  // TMEM lane
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t o_col = wg * 128, s_col = 256 + wg * 128, p_col = s_col + 64;
        const int m = wg * 128 + row;
        auto pv_done = [&](int g) { return wait_all(&o_done[wg], g & 1); };
        bool ok = true;
        int g = 0;
        Item I = item_of(min(static_cast<int>(blockIdx.x), nitems - 1)), next_item = I;
        for (int x = blockIdx.x; ok && x < nitems; x += gridDim.x, I = next_item) {
            const int pos = I.P + min(I.t0 + m / GQ, I.n - 1);  // this row's own key
            float m_used = -INFINITY, lsum = 0.f;
            for (int j = 0; j < I.ntiles; ++j, ++g) {
                ok = wait_all(&s_full[wg], g & 1);
                if (!ok) break;
                pa::tc::fence_after();
                const int j0 = I.base(j);
                uint32_t ph[32], pl[32];
                const float alpha =
                    softmax_tile(lane_base + s_col, &s_free[wg], lane, pos - j0,
                                 pos - p.window - j0, p.sinks - j0, p.qscale, m_used, lsum, ph, pl);
                if (j > 0) {  // PV of the previous tile must be done: P and O are free
                    ok = pv_done(g - 1);
                    if (!ok) break;
                    pa::tc::fence_after();
                    rescale_o<D>(lane_base + o_col, alpha);
                }
                // (each group does so before its own P; both write zeros)
                if (has_hidden_rows(I, p.sinks, j0))
                    zero_hidden_rows<D>(I, p.sinks, j0,
                                        skv + (g % NST) * 2 * Lay::T_BYTES + Lay::T_BYTES, row);
                put_p(lane_base + p_col, ph, pl);
                if (lane == 0) mbar_arrive(&p_full[wg]);
            }
            if (!ok) break;
            // (while the last PV runs:) where this lane writes its part of four
            // rows, NULL for rows past the request, and the next item
            __nv_bfloat16 *dst[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int mr = m - lane + k * 8 + lane / 4, t = I.t0 + mr / GQ;
                dst[k] = t < I.n ? p.out +
                                       (static_cast<size_t>(I.qs + t) * p.Hq + I.hk * GQ + mr % GQ) * D +
                                       (lane & 3) * 8
                                 : nullptr;
            }
            next_item = item_of(min(x + static_cast<int>(gridDim.x), nitems - 1));
            ok = pv_done(g - 1);  // PV of the item's last tile
            if (!ok) break;
            pa::tc::fence_after();
            // O / sum, rounded, through this warp's 2 KB of shared memory, so that
            // four lanes write 64 bytes of a row (a lane writing its own row in
            // 16-byte pieces took 5,000 cycles per item and held up the next
            // item's products)
            uint8_t *stage = smem + Lay::OFF_OUT + warp * 2048;
            auto swz = [](int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); };
            const float inv = 1.f / lsum;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t u[32];
                pa::tc::ld32(lane_base + o_col + c0, u);
                pa::tc::wait_ld();
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    auto pair = [&](int k) {
                        return pack_bf16(__uint_as_float(u[8 * c + k]) * inv,
                                         __uint_as_float(u[8 * c + k + 1]) * inv);
                    };
                    *reinterpret_cast<uint4 *>(stage + swz(lane, c)) =
                        make_uint4(pair(0), pair(2), pair(4), pair(6));
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 w4 = *reinterpret_cast<const uint4 *>(
                        stage + swz(k * 8 + lane / 4, lane & 3));
                    if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + c0) = w4;
                }
                __syncwarp();
            }
            // O of this group may be overwritten once every warp has read it
            pa::tc::fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[wg]);
        }
        if (!ok) *fail = 1;
    }

    // ---- tear-down ----------------------------------------------------------------
    pa::tc::fence_before();
    __syncthreads();
    if (*fail) {
        // a wait ran out: record it, then let the MMAs and the K/V copies in
        // flight land (bounded) before TMEM and shared memory go away
        if (tid == 0) pa::record_error(p.err, PA_DEVERR_TIMEOUT);
        if (warp == Lay::MMA_WARP || warp == Lay::MMA_WARP_B) {
            if (pa::tc::elect_one()) pa::tc::commit(drain);
            __syncwarp();
            (void)pa::mbar_wait(drain, 0);
        }
        if (warp == Lay::LOAD_WARP && lane == 0) {
            // the last tile issued into each stage
            for (int st = 0; st < NST && st < loads_issued; ++st) {
                const int g_last = st + NST * ((loads_issued - 1 - st) / NST);
                (void)pa::mbar_wait(&kv_full[st], (g_last / NST) & 1);
            }
        }
        pa::tc::fence_before();
        __syncthreads();
    }
    if (warp == Lay::MMA_WARP) {
        pa::tc::fence_after();
        pa::tc::dealloc(tmem, Lay::TMEM_COLS);
    }
}

// One query tile per cluster; see SLayout and the head of the file.
template <int D, int GQ>
__global__ void __launch_bounds__(SLayout<D>::THREADS, 1)
    prefill_window_split_kernel(const WinParams p, const __grid_constant__ CUtensorMap kmap,
                                const __grid_constant__ CUtensorMap vmap,
                                const __grid_constant__ CUtensorMap qmap) {
    using Lay = SLayout<D>;
    constexpr int NST = Lay::NST;
    constexpr int QTOK = 128 / GQ;  // query tokens per item
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sq = pa::smem_u32(smem), sk = sq + Lay::OFF_K, sv = sq + Lay::OFF_V;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *k_full = bars, *k_empty = k_full + NST, *v_full = k_empty + NST, *v_empty = v_full + NST;
    uint64_t *s_full = v_empty + NST, *s_free = s_full + 2;  // [group]
    uint64_t *p_full = s_free + 2, *o_done = p_full + 2, *q_full = o_done + 2, *drain = q_full + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_MISC);
    volatile int *fail = reinterpret_cast<volatile int *>(smem + Lay::OFF_MISC + 4);
    ReqTables &req = *reinterpret_cast<ReqTables *>(smem + Lay::OFF_REQ);
    uint32_t C, rank;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // ---- set-up: barriers, TMEM ------------------------------------------------
    if (tid == 0) {
        for (const CUtensorMap *map : {&kmap, &vmap, &qmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
        for (int i = 0; i < NST; ++i) {
            pa::mbar_init(&k_full[i], 1);
            pa::mbar_init(&k_empty[i], 1);
            pa::mbar_init(&v_full[i], 1);
            pa::mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            pa::mbar_init(&s_full[i], 1);
            pa::mbar_init(&s_free[i], 4);  // one arrival per softmax warp
            pa::mbar_init(&p_full[i], 4);
            pa::mbar_init(&o_done[i], 1);
        }
        pa::mbar_init(q_full, 1);
        pa::mbar_init(drain, 2);
        *fail = 0;
        pa::fence_barrier_init();
    }
    if (warp == Lay::MMA_WARP) pa::tc::alloc(tslot, Lay::TMEM_COLS);
    pa::tc::fence_before();
    __syncthreads();
    pa::tc::fence_after();
    const uint32_t tmem = *tslot;
    // launched as a programmatic dependent: the inputs are ready past this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int nitems = read_requests(p, req, QTOK) * p.Hkv;
    const int x = blockIdx.x / C;
    // (more items than clusters: the requests' rows overlap; the rest is left out)
    if (blockIdx.x == 0 && tid == 0 && nitems > static_cast<int>(gridDim.x / C))
        pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
    const bool idle = x >= nitems;  // the whole cluster
    const Item I = make_item(p, req, idle ? max(0, nitems - 1) : x, QTOK);
    // this CTA's tiles [ta, ta + nt) of the item; its i-th tile is group (i & 1)'s
    const int ta = idle ? 0 : static_cast<int>(int64_t(I.ntiles) * rank / C);
    const int nt = idle ? 0 : static_cast<int>(int64_t(I.ntiles) * (rank + 1) / C) - ta;

    int loads_issued = 0;  // a loader's lane 0: tiles issued (for the drain after a failure)
    const int wg = warp >> 2;   // softmax warps: group A or B
    const int row = tid & 127;  // and the row
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    float m_used = -INFINITY, lsum = 0.f;

    if (idle) {
        // no item: straight to the tear-down
    } else if (warp == Lay::K_WARP || warp == Lay::V_WARP) {
        // ---------------- loaders: K; the query tile, then V ----------------
        const bool is_v = warp == Lay::V_WARP;
        if (is_v && lane == 0) {
            // (rows past the request's new tokens affect nothing, as above)
            pa::mbar_arrive_expect_tx(q_full, Lay::QT_BYTES);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                tma_load_3d(sq + h * (128 * 128), &qmap, h * 64, I.hk * GQ, I.qs + I.t0, q_full);
        }
        __syncwarp();
        uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
        const CUtensorMap *map = is_v ? &vmap : &kmap;
        const uint32_t ring = is_v ? sv : sk;
        RowFetch rf(p, I, lane, ta, ta + nt);
        for (int i = 0; i < nt; ++i) {
            const int st = i % NST, slot0 = rf.advance(ta + i);
            if (i >= NST && !wait_all(&empty[st], ((i / NST) - 1) & 1)) {
                *fail = 1;
                break;
            }
            if (lane == 0) {
                pa::mbar_arrive_expect_tx(&full[st], Lay::T_BYTES);
                ++loads_issued;
            }
            __syncwarp();
            if (lane >= slot0 && lane < slot0 + rf.nb) {
                const uint32_t b = static_cast<uint32_t>(lane - slot0) * p.bs * 128;
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                    tma_load_2d(ring + st * Lay::T_BYTES + h * kT2KT * 128 + b, map, h * 64, rf.row,
                                &full[st]);
            }
            __syncwarp();
        }
        // the query tile must have landed before its place is used again
        if (is_v && !wait_all(q_full, 0)) *fail = 1;
    } else if (warp == Lay::MMA_WARP || warp == Lay::MMA_WARP_B) {
        // ---------------- MMA issuers, one per group ----------------
        const int g = warp == Lay::MMA_WARP ? 0 : 1;
        const uint64_t dq = pa::tc::sdesc(sq, 16, 1024);
        const uint64_t dk = pa::tc::sdesc(sk, 16, 1024), dv = pa::tc::sdesc(sv, kT2KT * 128, 1024);
        const uint32_t sc = tmem + 256 + g * 128, od = tmem + g * 128;
        constexpr uint32_t kStage = Lay::T_BYTES >> 4;
        // S of tile i, the group's l-th; its K is then free
        auto start = [&](int i, int l) {
            if (!wait_all(&k_full[i % NST], (i / NST) & 1)) return false;
            if (l > 0 && !wait_all(&s_free[g], (l - 1) & 1)) return false;
            pa::tc::fence_after();
            if (pa::tc::elect_one()) {
                mma_s<D>(sc, dq, dk + static_cast<uint32_t>((i % NST) * kStage));
                pa::tc::commit(&s_full[g]);
                pa::tc::commit(&k_empty[i % NST]);
            }
            __syncwarp();
            return true;
        };
        bool ok = g < nt ? wait_all(q_full, 0) && start(g, 0) : true;
        for (int i = g, l = 0; i < nt && ok; i += 2, ++l) {
            if (i + 2 < nt) ok = start(i + 2, l + 1);
            if (ok) ok = wait_all(&v_full[i % NST], (i / NST) & 1) && wait_all(&p_full[g], l & 1);
            if (!ok) break;
            pa::tc::fence_after();
            if (pa::tc::elect_one()) {
                mma_pv<D>(od, sc + 64, dv + static_cast<uint32_t>((i % NST) * kStage), l > 0);
                pa::tc::commit(&o_done[g]);
                pa::tc::commit(&v_empty[i % NST]);
            }
            __syncwarp();
        }
        if (!ok) *fail = 1;
    } else {
        // ---------------- softmax warp groups ----------------
        const int pos = I.P + min(I.t0 + row / GQ, I.n - 1);  // this row's own key
        const uint32_t o_col = wg * 128, s_col = 256 + wg * 128, p_col = s_col + 64;
        auto pv_done = [&](int l) { return wait_all(&o_done[wg], l & 1); };
        bool ok = true;
        int l = 0;
        for (int i = wg; i < nt; i += 2, ++l) {
            ok = wait_all(&s_full[wg], l & 1);
            if (!ok) break;
            pa::tc::fence_after();
            const int j0 = I.base(ta + i);
            uint32_t ph[32], pl[32];
            const float alpha =
                softmax_tile(lane_base + s_col, &s_free[wg], lane, pos - j0, pos - p.window - j0,
                             p.sinks - j0, p.qscale, m_used, lsum, ph, pl);
            if (l > 0) {  // PV of the previous tile must be done: P and O are free
                ok = pv_done(l - 1);
                if (!ok) break;
                pa::tc::fence_after();
                rescale_o<D>(lane_base + o_col, alpha);
            }
            if (has_hidden_rows(I, p.sinks, j0)) {
                ok = wait_all(&v_full[i % NST], (i / NST) & 1);  // V has landed
                if (!ok) break;
                zero_hidden_rows<D>(I, p.sinks, j0, sv + (i % NST) * Lay::T_BYTES, row);
            }
            put_p(lane_base + p_col, ph, pl);
            if (lane == 0) mbar_arrive(&p_full[wg]);
        }
        if (ok && l > 0) ok = pv_done(l - 1);
        pa::tc::fence_after();
        if (!ok) *fail = 1;
    }

    // ---- the cluster's results ------------------------------------------------------
    // Every warp of the cluster comes here: its products are done and its tiles
    // have been used, so the rings and the query tile may be written.
    auto cluster_sync = [] {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    };
    __syncwarp();
    if (C > 1) cluster_sync();
    else __syncthreads();
    auto at = [](uint32_t addr, uint32_t cta) {
        uint32_t r;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
        return r;
    };
    const int cols = D / C;  // columns that a CTA finishes: 16 or more
    const int t = I.t0 + row / GQ;
    __nv_bfloat16 *dst = p.out + (static_cast<size_t>(I.qs + min(t, I.n - 1)) * p.Hq + I.hk * GQ +
                                  row % GQ) * D;
    float2 *ml = reinterpret_cast<float2 *>(smem), *xml = ml + Lay::MAX_C * 128;
    if (!idle && warp < 8) {
        // The two groups first: each takes half of the columns, gives the other
        // its part of the other half, and sums what it has to its own weights.
        float4 *xs = reinterpret_cast<float4 *>(smem + Lay::OFF_K + Lay::X_BYTES);
        const bool any = wg < nt;  // this group had a tile
        const uint32_t o_addr = lane_base + wg * 128;
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2; c0 += 16) {
            uint32_t u[16];
            pa::tc::ld16(o_addr + (wg ^ 1) * (D / 2) + c0, u);
            pa::tc::wait_ld();
#pragma unroll
            for (int k = 0; k < 4; ++k)
                xs[(wg * (D / 8) + c0 / 4 + k) * 128 + row] =
                    make_float4(__uint_as_float(u[4 * k]), __uint_as_float(u[4 * k + 1]),
                                __uint_as_float(u[4 * k + 2]), __uint_as_float(u[4 * k + 3]));
        }
        xml[wg * 128 + row] = make_float2(m_used, lsum);
        asm volatile("bar.sync 1, 256;" ::: "memory");  // the eight softmax warps
        const float2 other = xml[(wg ^ 1) * 128 + row];
        const float M = fmaxf(m_used, other.x);
        const float fm = m_used == -INFINITY ? 0.f : exp2f(m_used - M);
        const float fo = other.x == -INFINITY ? 0.f : exp2f(other.x - M);
        const float l = lsum * fm + other.y * fo;
        const bool any_other = (wg ^ 1) < nt;
        const float inv = C == 1 ? 1.f / l : 1.f;
        // rows past the request's tokens travel only with one that is not
        const bool wanted = __any_sync(pa::kFull, t < I.n);
#pragma unroll 1
        for (int c0 = 0; c0 < D / 2 && wanted; c0 += 16) {
            uint32_t u[16];
            pa::tc::ld16(o_addr + wg * (D / 2) + c0, u);
            pa::tc::wait_ld();
            float o[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 v = xs[((wg ^ 1) * (D / 8) + c0 / 4 + k) * 128 + row];
                const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[4 * k + e] = ((any ? __uint_as_float(u[4 * k + e]) * fm : 0.f) +
                                    (any_other ? vv[e] * fo : 0.f)) * inv;
            }
            const int c = wg * (D / 2) + c0;
            if (C == 1) {
                if (t < I.n) {
#pragma unroll
                    for (int k = 0; k < 16; k += 8)
                        *reinterpret_cast<uint4 *>(dst + c + k) = make_uint4(
                            pack_bf16(o[k], o[k + 1]), pack_bf16(o[k + 2], o[k + 3]),
                            pack_bf16(o[k + 4], o[k + 5]), pack_bf16(o[k + 6], o[k + 7]));
                }
            } else {
                const uint32_t to = at(sk + ((rank * (cols / 4) + c % cols / 4) * 128 + row) * 16, c / cols);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(to + k * 128 * 16),
                                 "f"(o[4 * k]), "f"(o[4 * k + 1]), "f"(o[4 * k + 2]), "f"(o[4 * k + 3])
                                 : "memory");
            }
        }
        if (wg == 0 && C > 1)
            for (uint32_t to = 0; to < C; ++to)
                asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(
                                 at(sq + (rank * 128 + row) * 8, to)),
                             "f"(M), "f"(l)
                             : "memory");
        pa::tc::fence_before();
    }
    __syncwarp();
    if (C > 1) cluster_sync();  // nothing is sent after this: a CTA may exit before the others
    if (!idle && warp < 8 && C > 1 && t < I.n) {
        const float4 *xs = reinterpret_cast<const float4 *>(smem + Lay::OFF_K);
        float w[Lay::MAX_C], M = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < Lay::MAX_C; ++k)
            if (k < C) M = fmaxf(M, ml[k * 128 + row].x);
#pragma unroll
        for (int k = 0; k < Lay::MAX_C; ++k) {
            w[k] = 0.f;
            if (k < C) {
                const float2 v = ml[k * 128 + row];
                w[k] = v.x == -INFINITY ? 0.f : exp2f(v.x - M);  // 0 for a CTA that saw nothing
                l += w[k] * v.y;
            }
        }
        const float inv = 1.f / l;
        // group A's threads finish the first half of the CTA's columns, B's the second
        for (int c = wg * (cols / 2); c < (wg + 1) * (cols / 2); c += 8) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
#pragma unroll
            for (int k = 0; k < Lay::MAX_C; ++k) {
                if (k >= C) break;
                const float f = w[k];
                const float4 u = xs[(k * (cols / 4) + c / 4) * 128 + row];
                const float4 v = xs[(k * (cols / 4) + c / 4 + 1) * 128 + row];
                a.x = fmaf(f, u.x, a.x), a.y = fmaf(f, u.y, a.y);
                a.z = fmaf(f, u.z, a.z), a.w = fmaf(f, u.w, a.w);
                b.x = fmaf(f, v.x, b.x), b.y = fmaf(f, v.y, b.y);
                b.z = fmaf(f, v.z, b.z), b.w = fmaf(f, v.w, b.w);
            }
            *reinterpret_cast<uint4 *>(dst + rank * cols + c) =
                make_uint4(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv),
                           pack_bf16(b.x * inv, b.y * inv), pack_bf16(b.z * inv, b.w * inv));
        }
    }

    // ---- tear-down ----------------------------------------------------------------
    __syncthreads();
    if (*fail) {
        // a wait ran out: record it, then let the MMAs and the copies in flight
        // land (bounded) before TMEM and shared memory go away
        if (tid == 0) pa::record_error(p.err, PA_DEVERR_TIMEOUT);
        if (warp == Lay::MMA_WARP || warp == Lay::MMA_WARP_B) {
            if (pa::tc::elect_one()) pa::tc::commit(drain);
            __syncwarp();
            (void)pa::mbar_wait(drain, 0);
        }
        if ((warp == Lay::K_WARP || warp == Lay::V_WARP) && lane == 0) {
            uint64_t *full = warp == Lay::V_WARP ? v_full : k_full;
            for (int st = 0; st < NST && st < loads_issued; ++st) {
                const int last = st + NST * ((loads_issued - 1 - st) / NST);
                (void)pa::mbar_wait(&full[st], (last / NST) & 1);
            }
        }
        __syncthreads();
    }
    if (warp == Lay::MMA_WARP) {
        pa::tc::fence_after();
        pa::tc::dealloc(tmem, Lay::TMEM_COLS);
    }
}

// Upper bound of the query tiles of qtok tokens: at most one per request is
// partly filled.
int64_t query_tiles(int R, int T, int max_query_len, int qtok) {
    return std::min<int64_t>(int64_t(R) * ((int64_t(max_query_len) + qtok - 1) / qtok),
                             int64_t(T) / qtok + R);
}

// Whether a call runs on the split kernel: its (query tile of 128 rows, KV
// head) pairs, returned in *singles, fit one per SM.
bool runs_split(int R, int T, int max_query_len, int gq, int Hkv, int sms, int64_t *singles) {
    *singles = query_tiles(R, T, max_query_len, 128 / gq) * Hkv;
    return R <= kMaxR && *singles <= sms;
}

// SMs of the current device; 0: a CUDA call failed.
int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

// Launches kernel `kern` for groups of at most kMaxR requests, its tables' size;
// ctas(p): the grid of a launch.
template <int D, int GQ, typename K, typename F>
int launch_all(K kern, int threads, size_t smem, int cluster, const WinParams &p0, const void *q,
               const void *k_cache, const void *v_cache, F &&ctas, cudaStream_t stream) {
    const int64_t rows = (p0.num_blocks * p0.Hkv) << p0.bs_log2;
    CUtensorMap kmap, vmap, qmap;
    const int box = std::min(p0.bs, kT2KT);
    if (int rc = pa::encode_pool_map(&kmap, k_cache, rows, D, box)) return rc;
    if (int rc = pa::encode_pool_map(&vmap, v_cache, rows, D, box)) return rc;
    if (int rc = pa::encode_q_map(&qmap, q, p0.T, p0.Hq, D, GQ, 128 / GQ)) return rc;
    for (int r0 = 0; r0 < p0.R; r0 += kMaxR) {
        WinParams p = p0;
        p.R = std::min(kMaxR, p0.R - r0);
        p.block_table += int64_t(r0) * p.MB;
        p.query_start += r0;
        p.context_lens += r0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(ctas(p)));
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = cluster > 0 ? 2 : 1;
        (void)cudaGetLastError();  // drop a stale error that is not ours
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, kmap, vmap, qmap);
        if (e != cudaSuccess) return pa::cuda_fail(e, "prefill_window launch");
        if (int rc = pa::check_launch("prefill_window launch")) return rc;
    }
    return PA_OK;
}

template <int D, int GQ>
int launch(const WinParams &p, const void *q, const void *k_cache, const void *v_cache,
           int max_query_len, cudaStream_t stream) {
    const int sms = sm_count();
    if (sms <= 0) return pa::cuda_fail(cudaGetLastError(), "prefill_window: SM count");
    int64_t singles = 0;
    if (runs_split(p.R, p.T, max_query_len, GQ, p.Hkv, sms, &singles)) {
        auto kern = prefill_window_split_kernel<D, GQ>;
        static std::atomic<uint64_t> done{0};
        if (int rc = set_smem_once(kern, SLayout<D>::SMEM, &done)) return rc;
        // Clusters as large as run at once, with a K/V tile for each group.  8 KV
        // heads, d 128: 40 tokens with window 4096 68 us on the kernel above, 44 as
        // one CTA per query tile, 26.7 in two waves of clusters of 8, 18.0 in one of
        // 4; 64 tokens of d 64 with that window 60.8, 34.7 and (clusters of 4)
        // 13.8 us; 256 tokens of window 1024 24.3, 17.6 and (of 2) 13.6 us.
        static std::atomic<int> cache[64][5];
        const int64_t keys = std::min<int64_t>(int64_t(p.MB) << p.bs_log2,
                                               int64_t(p.window) + p.sinks + 128 / GQ);
        int c = 1;
        while (2 * c <= SLayout<D>::MAX_C && keys >= 4 * c * kT2KT) {
            const int n = clusters_at_once(kern, SLayout<D>::THREADS, SLayout<D>::SMEM, 2 * c, cache);
            if (n < 0) return pa::cuda_fail(cudaGetLastError(), "prefill_window: occupancy");
            if (singles > n) break;
            c *= 2;
        }
        return launch_all<D, GQ>(kern, SLayout<D>::THREADS, SLayout<D>::SMEM, c, p, q, k_cache, v_cache,
                                 [&](const WinParams &) { return singles * c; }, stream);
    }
    auto kern = prefill_window_kernel<D, GQ>;
    static std::atomic<uint64_t> done{0};
    if (int rc = set_smem_once(kern, WLayout<D>::SMEM, &done)) return rc;
    return launch_all<D, GQ>(
        kern, WLayout<D>::THREADS, WLayout<D>::SMEM, 0, p, q, k_cache, v_cache,
        [&](const WinParams &pp) {
            return std::max<int64_t>(
                1, std::min<int64_t>(sms, query_tiles(pp.R, pp.T, max_query_len, 256 / GQ) * pp.Hkv));
        },
        stream);
}

}  // namespace

extern "C" int pa_prefill_window(void *out, const void *q, const void *k_cache,
                                 const void *v_cache, const int32_t *block_table,
                                 int max_blocks_per_seq, const int32_t *query_start,
                                 const int32_t *context_lens, int R, int total_tokens,
                                 int max_query_len, int Hq, int Hkv, int head_dim, int block_size,
                                 int64_t num_blocks, float scale, int window, int num_sinks,
                                 int dtype, pa_stream_t stream) {
    pa::clear_error();
    if (dtype != PA_BF16)
        return pa::fail(dtype == PA_F32 ? PA_ERR_UNSUPPORTED : PA_ERR_INVALID,
                        "prefill_window: bf16 only");
    if (R < 0 || total_tokens < 0 || max_query_len < 0 || Hq <= 0 || Hkv <= 0 || Hkv > 1024 ||
        Hq % Hkv || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return pa::fail(PA_ERR_INVALID, "prefill_window: bad sizes");
    if (head_dim != 64 && head_dim != 128)
        return pa::fail(PA_ERR_UNSUPPORTED, "prefill_window: head_dim %d unsupported", head_dim);
    const int gq = Hq / Hkv;
    if (gq != 1 && gq != 2 && gq != 4 && gq != 8)
        return pa::fail(PA_ERR_UNSUPPORTED, "prefill_window: Hq/Hkv=%d unsupported", gq);
    if (!pa::pow2_in(block_size, 8, 128))
        return pa::fail(PA_ERR_UNSUPPORTED, "prefill_window: block_size %d unsupported", block_size);
    if (int64_t(max_blocks_per_seq) * block_size > (int64_t(1) << 30))
        return pa::fail(PA_ERR_INVALID, "prefill_window: table capacity too large");
    if (num_blocks > INT32_MAX || num_blocks * Hkv * block_size > int64_t(INT32_MAX) - 256)
        return pa::fail(PA_ERR_UNSUPPORTED, "prefill_window: pools of 2^31 rows or more");
    // items are counted in 32 bits: (tokens / 16 + requests) * KV heads
    if ((int64_t(total_tokens) / 16 + std::min(R, kMaxR)) * Hkv > INT32_MAX / 2)
        return pa::fail(PA_ERR_UNSUPPORTED, "prefill_window: too many query tokens");
    if (window < 1 || num_sinks < 0)
        return pa::fail(PA_ERR_INVALID, "prefill_window: window %d must be positive, num_sinks %d "
                                        "not negative", window, num_sinks);
    if (!(scale > 0.f) || !std::isfinite(scale))
        return pa::fail(PA_ERR_INVALID, "prefill_window: scale must be positive and finite");
    if (R == 0 || total_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_table || !query_start || !context_lens)
        return pa::fail(PA_ERR_INVALID, "prefill_window: NULL pointer");
    if (!pa::aligned16(q) || !pa::aligned16(out) || !pa::aligned16(k_cache) ||
        !pa::aligned16(v_cache))
        return pa::fail(PA_ERR_INVALID, "prefill_window: q, out and pools must be 16-byte aligned");
    if (pa::validate_on())
        if (int rc = pa::validate_window(block_table, max_blocks_per_seq, context_lens, query_start,
                                         total_tokens, max_query_len, R, block_size, num_blocks,
                                         window, num_sinks, stream))
            return rc;
    WinParams p{};
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.block_table = block_table;
    p.query_start = query_start;
    p.context_lens = context_lens;
    p.err = pa::device_error_word();
    p.num_blocks = num_blocks;
    p.R = R;
    p.T = total_tokens;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.bs = block_size;
    p.bs_log2 = log2_int(block_size);
    p.MB = max_blocks_per_seq;
    // contexts have at most 2^30 tokens: a wider window or more sinks show no more
    p.window = std::min(window, 1 << 30);
    p.sinks = std::min(num_sinks, 1 << 30);
    p.qscale = scale * kLog2e;
    auto pick = [&](auto d) -> int {
        constexpr int DD = decltype(d)::value;
        switch (gq) {
            case 1: return launch<DD, 1>(p, q, k_cache, v_cache, max_query_len, stream);
            case 2: return launch<DD, 2>(p, q, k_cache, v_cache, max_query_len, stream);
            case 4: return launch<DD, 4>(p, q, k_cache, v_cache, max_query_len, stream);
            default: return launch<DD, 8>(p, q, k_cache, v_cache, max_query_len, stream);
        }
    };
    return head_dim == 128 ? pick(std::integral_constant<int, 128>{})
                           : pick(std::integral_constant<int, 64>{});
}

extern "C" int pa_prefill_window_kernel_for(int R, int total_tokens, int max_query_len, int Hq, int Hkv,
                                            int *kernel) {
    pa::clear_error();
    if (!kernel) return pa::fail(PA_ERR_INVALID, "prefill_window_kernel_for: kernel is NULL");
    if (R < 0 || total_tokens < 0 || max_query_len < 0 || Hq <= 0 || Hkv <= 0 || Hkv > 1024 || Hq % Hkv)
        return pa::fail(PA_ERR_INVALID, "prefill_window_kernel_for: bad sizes");
    const int gq = Hq / Hkv;
    if (gq != 1 && gq != 2 && gq != 4 && gq != 8)
        return pa::fail(PA_ERR_UNSUPPORTED, "prefill_window_kernel_for: Hq/Hkv=%d unsupported", gq);
    const int sms = sm_count();
    if (sms <= 0) return pa::cuda_fail(cudaGetLastError(), "prefill_window_kernel_for: SM count");
    int64_t singles = 0;
    *kernel = runs_split(R, total_tokens, max_query_len, gq, Hkv, sms, &singles)
                  ? PA_PREFILL_WINDOW_SPLIT
                  : PA_PREFILL_WINDOW_PERSISTENT;
    return PA_OK;
}
