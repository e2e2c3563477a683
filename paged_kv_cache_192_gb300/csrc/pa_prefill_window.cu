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
// The groups share an item in one of two ways.  With many items, A and B are
// its two query tiles of 128 rows and both use every K/V tile.  With few
// (SPLIT), an item is one query tile: A takes the even K/V tiles and B the odd
// ones, and the two results meet through shared memory by log-sum-exp, so that
// an item takes half as long and twice as many SMs have one.
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

template <int D>
struct WLayout {
    static constexpr int NST = 4;
    static constexpr int THREADS = 12 * 32;
    static constexpr int MMA_WARP = 8, LOAD_WARP = 9, Q_WARP = 10, MMA_WARP_B = 11;
    static constexpr int TMEM_COLS = 512;
    static constexpr int QT_BYTES = 128 * D * 2;   // one query tile
    static constexpr int T_BYTES = kT2KT * D * 2;  // one K or V tile
    static constexpr int OFF_X = QT_BYTES;         // second query tile; SPLIT: exchange of O
    static constexpr int OFF_KV = 2 * QT_BYTES;    // [stage][K|V]
    static constexpr int OFF_BAR = OFF_KV + NST * 2 * T_BYTES;
    // kv_full, kv_empty [NST]; s_full, s_free, p_full, o_done, o_free, x_full
    // [2]; q_full, q_empty, drain
    static constexpr int N_BAR = 2 * NST + 12 + 3;
    static constexpr int OFF_MISC = OFF_BAR + 8 * N_BAR;   // TMEM slot, fail flag, scan scratch
    static constexpr int OFF_ML = OFF_MISC + 64;           // SPLIT: (max, sum) [2][128]
    static constexpr int OFF_PRE = OFF_ML + 2 * 128 * 8;   // [kMaxR + 1] query tiles before request r
    static constexpr int OFF_QS = OFF_PRE + 4 * (kMaxR + 1);
    static constexpr int OFF_N = OFF_QS + 4 * kMaxR;
    static constexpr int OFF_L = OFF_N + 4 * kMaxR;
    static constexpr int OFF_OUT = (OFF_L + 4 * kMaxR + 15) / 16 * 16;  // staged output, 2 KB per warp
    static constexpr int SMEM = OFF_OUT + 8 * 2048 + 1024;
    static_assert(OFF_BAR % 8 == 0 && OFF_ML % 8 == 0 && OFF_X % 16 == 0, "alignment");
    static_assert(QT_BYTES >= 128 * (D / 2) * 4, "half of O must fit the exchange");
    static_assert(SMEM <= 227 * 1024, "shared memory");
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

template <int D, int GQ, bool SPLIT>
__global__ void __launch_bounds__(WLayout<D>::THREADS, 1)
    prefill_window_kernel(const WinParams p, const __grid_constant__ CUtensorMap kmap,
                          const __grid_constant__ CUtensorMap vmap,
                          const __grid_constant__ CUtensorMap qmap) {
    using Lay = WLayout<D>;
    constexpr int NST = Lay::NST;
    constexpr int CH = D * 2 / 16;  // 16-byte chunks per row
    constexpr int QTILES = SPLIT ? 1 : 2;     // query tiles per item
    constexpr int STEP = SPLIT ? 2 : 1;       // K/V tiles from one of a group to its next
    constexpr int QTOK = QTILES * 128 / GQ;   // query tokens per item
    constexpr int TILE_TX = 2 * kT2KT * D * 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sq = pa::smem_u32(smem), skv = sq + Lay::OFF_KV;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR);
    uint64_t *kv_full = bars, *kv_empty = bars + NST;
    uint64_t *s_full = bars + 2 * NST, *s_free = s_full + 2;  // [group]
    uint64_t *p_full = s_free + 2, *o_done = p_full + 2, *o_free = o_done + 2;
    uint64_t *x_full = o_free + 2;  // [group that wrote]
    uint64_t *q_full = x_full + 2, *q_empty = q_full + 1, *drain = q_empty + 1;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + Lay::OFF_MISC);
    volatile int *fail = reinterpret_cast<volatile int *>(smem + Lay::OFF_MISC + 4);
    int *scan = reinterpret_cast<int *>(smem + Lay::OFF_MISC + 8);  // [12]
    int *pre = reinterpret_cast<int *>(smem + Lay::OFF_PRE);
    int *req_qs = reinterpret_cast<int *>(smem + Lay::OFF_QS);
    int *req_n = reinterpret_cast<int *>(smem + Lay::OFF_N);
    int *req_L = reinterpret_cast<int *>(smem + Lay::OFF_L);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // ---- set-up: barriers, TMEM ------------------------------------------------
    if (tid == 0) {
        for (const CUtensorMap *map : {&kmap, &vmap, &qmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
        for (int i = 0; i < NST; ++i) {
            pa::mbar_init(&kv_full[i], 1);
            pa::mbar_init(&kv_empty[i], SPLIT ? 1 : 2);  // the PV of the groups that use it
        }
        for (int i = 0; i < 2; ++i) {
            pa::mbar_init(&s_full[i], 1);
            pa::mbar_init(&s_free[i], 4);  // one arrival per softmax warp
            pa::mbar_init(&p_full[i], 4);
            pa::mbar_init(&o_done[i], 1);
            pa::mbar_init(&o_free[i], 4);
            pa::mbar_init(&x_full[i], 4);
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

    // ---- the requests and the prefix sum of their query tiles --------------------
    int carry = 0;
    for (int r0 = 0; r0 < p.R; r0 += Lay::THREADS) {
        const int r = r0 + tid;
        int np = 0;
        if (r < p.R) {
            const int qs = p.query_start[r], n = p.query_start[r + 1] - qs, L = p.context_lens[r];
            if (n > 0 && qs >= 0 && n <= p.T - qs && L >= n && L <= p.MB << p.bs_log2)
                np = (n + QTOK - 1) / QTOK;
            else if (n != 0 || L < 0 || L > p.MB << p.bs_log2)
                pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
            req_qs[r] = qs;
            req_n[r] = n;
            req_L[r] = L;
        }
        int x = np;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(pa::kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan[warp] = x;
        __syncthreads();
        int off = carry;
        for (int w = 0; w < Lay::THREADS / 32; ++w) {
            off += w < warp ? scan[w] : 0;
            carry += scan[w];
        }
        if (r < p.R) pre[r + 1] = off + x;
        __syncthreads();
    }
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const int nitems = carry * p.Hkv;

    auto item_of = [&](int x) {
        Item it;
        const int pair = x / p.Hkv;
        it.hk = x % p.Hkv;
        int lo = 0, hi = p.R - 1;  // the last request with pre[r] <= pair
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= pair) lo = mid;
            else hi = mid - 1;
        }
        it.r = lo;
        // the last query tiles first: they see the most keys
        it.t0 = (pre[lo + 1] - 1 - pair) * QTOK;
        it.qs = req_qs[lo];
        it.n = req_n[lo];
        it.P = req_L[lo] - it.n;
        it.kv_end = min(it.P + it.n, it.P + it.t0 + QTOK);
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
    };

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
            if (it > 0 && !__all_sync(pa::kFull, pa::mbar_wait(q_empty, (it - 1) & 1))) {
                *fail = 1;
                break;
            }
            if (lane == 0) {
                pa::mbar_arrive_expect_tx(q_full, QTILES * Lay::QT_BYTES);
                for (int qt = 0; qt < QTILES; ++qt)
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
        const int rows_total = static_cast<int>(p.num_blocks * p.Hkv) << p.bs_log2;
        const int nb = max(1, kT2KT >> p.bs_log2), tpb = 32 / nb;  // blocks per tile, tiles per batch
        int g = 0;  // CTA-wide K/V tile counter
        for (int x = blockIdx.x; x < nitems && !*fail; x += gridDim.x) {
            const Item I = item_of(x);
            const int32_t *bt = p.block_table + static_cast<size_t>(I.r) * p.MB;
            // pool row of this lane's (tile, block) slot of the batch from tile tb on;
            // a block that no row sees is out of bounds: zero-filled, not read
            auto fetch = [&](int tb) -> int {
                const int j = tb + lane / nb;
                if (j >= I.ntiles) return rows_total;
                const int tok = I.base(j) + (lane % nb) * p.bs;
                const int blk0 = tok & ~(p.bs - 1);  // (blocks of 128: the tile is half of one)
                if (tok >= I.kv_end || (tok >= p.sinks && blk0 + p.bs <= I.lo)) return rows_total;
                int v = __ldg(bt + (tok >> p.bs_log2));
                if (v < 0 || v >= p.num_blocks) {
                    pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
                    v = 0;
                }
                return ((v * p.Hkv + I.hk) << p.bs_log2) + (tok & (p.bs - 1));
            };
            int row = fetch(0), row_next = fetch(tpb), tb = 0;
            bool ok = true;
            for (int j = 0; j < I.ntiles && ok; ++j, ++g) {
                if (j - tb >= tpb) {
                    tb += tpb;
                    row = row_next;
                    row_next = fetch(tb + tpb);
                }
                const int st = g % NST, slot0 = (j - tb) * nb;
                if (g >= NST) ok = __all_sync(pa::kFull, pa::mbar_wait(&kv_empty[st], ((g / NST) - 1) & 1));
                if (!ok) break;
                const uint32_t kst = skv + st * 2 * Lay::T_BYTES, vst = kst + Lay::T_BYTES;
                if (lane == 0) {
                    pa::mbar_arrive_expect_tx(&kv_full[st], TILE_TX);
                    ++loads_issued;
                }
                __syncwarp();
                // the lane that holds a block's row issues its copies
                if (lane >= slot0 && lane < slot0 + nb) {
                    const uint32_t b = static_cast<uint32_t>(lane - slot0) * p.bs * 128;
#pragma unroll
                    for (int h = 0; h < D / 64; ++h) {
                        const uint32_t off = h * kT2KT * 128 + b;
                        tma_load_2d(kst + off, &kmap, h * 64, row, &kv_full[st]);
                        tma_load_2d(vst + off, &vmap, h * 64, row, &kv_full[st]);
                    }
                }
                __syncwarp();
            }
            if (!ok) *fail = 1;
        }
    } else if (warp == Lay::MMA_WARP || warp == Lay::MMA_WARP_B) {
        // ---------------- MMA issuers, one per group ----------------
        const int wg = warp == Lay::MMA_WARP ? 0 : 1;
        constexpr uint32_t kIdS = pa::tc::idesc_bf16(128, kT2KT, 0, 0);
        constexpr uint32_t kIdO = pa::tc::idesc_bf16(128, D, 0, 1);
        constexpr uint32_t kStage = (2 * Lay::T_BYTES) >> 4;
        const uint64_t dq = pa::tc::sdesc(sq, 16, 1024) +
                            static_cast<uint32_t>(SPLIT ? 0 : wg * (Lay::QT_BYTES >> 4));
        const uint64_t dk = pa::tc::sdesc(skv, 16, 1024);
        const uint64_t dv = pa::tc::sdesc(skv + Lay::T_BYTES, kT2KT * 128, 1024);
        const uint32_t sc = tmem + 256 + wg * 128, ph = sc + 64, pl = ph + 32;
        const uint32_t od = tmem + wg * 128;
        auto wait_all = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(pa::kFull, pa::mbar_wait(bar, parity));
        };
        // S of CTA tile g, the group's l-th, once the group has loaded the last
        auto issue_s = [&](int g, int l) {
            if (l > 0 && !wait_all(&s_free[wg], (l - 1) & 1)) return false;
            pa::tc::fence_after();
            const uint64_t b0 = dk + static_cast<uint32_t>((g % NST) * kStage);
            if (pa::tc::elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    pa::tc::mma_ss(sc, dq + (((ks >> 2) * 128 * 128 + (ks & 3) * 32) >> 4),
                                   b0 + (((ks >> 2) * kT2KT * 128 + (ks & 3) * 32) >> 4), kIdS,
                                   ks > 0);
                pa::tc::commit(&s_full[wg]);
            }
            __syncwarp();
            return true;
        };
        // O (+)= P_hi V + P_lo V
        auto issue_pv = [&](int g, int acc0) {
            const uint64_t b0 = dv + static_cast<uint32_t>((g % NST) * kStage);
            if (pa::tc::elect_one()) {
#pragma unroll
                for (int ks = 0; ks < kT2KT / 16; ++ks) {
                    const uint64_t b = b0 + ((ks * 16 * 128) >> 4);
                    pa::tc::mma_ts(od, ph + ks * 8, b, kIdO, ks == 0 ? acc0 : 1);
                    pa::tc::mma_ts(od, pl + ks * 8, b, kIdO, 1);
                }
                pa::tc::commit(&o_done[wg]);
                pa::tc::commit(&kv_empty[g % NST]);
            }
            __syncwarp();
        };
        bool ok = true;
        int g0 = 0, l = 0, it = 0;  // CTA tiles before the item, tiles of the group so far
        for (int x = blockIdx.x; ok && x < nitems; x += gridDim.x, ++it) {
            const int nt = item_of(x).ntiles;
            ok = wait_all(q_full, it & 1);
            const int first = SPLIT ? wg : 0;
            auto start = [&](int j, int lj) {  // S of the item's tile j once its K has landed
                const int g = g0 + j;
                if (!wait_all(&kv_full[g % NST], (g / NST) & 1)) return false;
                pa::tc::fence_after();
                return issue_s(g, lj);
            };
            if (ok && first < nt) ok = start(first, l);
            for (int j = first; j < nt && ok; j += STEP, ++l) {
                if (j + STEP < nt) {
                    ok = start(j + STEP, l + 1);
                    if (!ok) break;
                } else {
                    if (pa::tc::elect_one()) pa::tc::commit(q_empty);
                    __syncwarp();
                }
                // the item's first PV overwrites O once the group has read the last item's
                if (j == first && it > 0) ok = wait_all(&o_free[wg], (it - 1) & 1);
                if (ok) ok = wait_all(&p_full[wg], l & 1);
                if (!ok) break;
                pa::tc::fence_after();
                issue_pv(g0 + j, j > first);
            }
            if (first >= nt) {  // no tile for this group: the query tile is free for its part
                if (pa::tc::elect_one()) pa::tc::commit(q_empty);
                __syncwarp();
            }
            g0 += nt;
        }
        if (!ok) *fail = 1;
    } else {
        // ---------------- softmax warp groups ----------------
        const int wg = warp >> 2;   // group A or B
        const int row = tid & 127;  // TMEM lane
        const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t o_col = wg * 128, s_col = 256 + wg * 128, p_col = s_col + 64;
        const int m = (SPLIT ? 0 : wg * 128) + row;
        const float qs2 = p.qscale;  // softmax scale in log2 units
        auto pv_done = [&](int l) { return pa::mbar_wait(&o_done[wg], l & 1); };
        bool ok = true;
        int g0 = 0, l = 0, it = 0;  // CTA tiles before the item, tiles of the group so far
        Item I = item_of(min(static_cast<int>(blockIdx.x), nitems - 1)), next_item = I;
        for (int x = blockIdx.x; ok && x < nitems; x += gridDim.x, ++it, I = next_item) {
            const int pos = I.P + min(I.t0 + m / GQ, I.n - 1);  // this row's own key
            float m_used = -INFINITY, lsum = 0.f;
            const int first = SPLIT ? wg : 0;
            for (int j = first; j < I.ntiles; j += STEP, ++l) {
                ok = pa::mbar_wait(&s_full[wg], l & 1);
                if (!ok) break;
                pa::tc::fence_after();
                uint32_t sr[2][32];
                pa::tc::ld32(lane_base + s_col, sr[0]);
                pa::tc::ld32(lane_base + s_col + 32, sr[1]);
                pa::tc::wait_ld();
                // S may now be overwritten by the next tile's
                pa::tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s_free[wg]);
                const int j0 = I.base(j);
                float s[64];
#pragma unroll
                for (int c = 0; c < 64; ++c) s[c] = __uint_as_float(sr[c >> 5][c & 31]);
                // hidden: keys past the row's own, and keys [S, pos - W]
                const int hi = pos - j0, wl = pos - p.window - j0, s0 = p.sinks - j0;
                if (hi < kT2KT - 1 || (wl >= 0 && s0 < kT2KT)) {
                    // bit c: key j0 + c is hidden; up(n): the bits from n on
                    auto up = [](int n) { return n >= 64 ? 0ull : ~0ull << max(n, 0); };
                    const uint64_t hidden = up(hi + 1) | (up(s0) & ~up(wl + 1));
                    const uint32_t hl = static_cast<uint32_t>(hidden),
                                   hh = static_cast<uint32_t>(hidden >> 32);
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
                uint32_t ph[32], pl[32];
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
                    const float2 lo = pa::ffma2(pa::bf16x2_to_float2(ph[c]),
                                                make_float2(-1.f, -1.f), make_float2(p0, p1));
                    pl[c] = pack_bf16(lo.x, lo.y);
                }
                const float rs = ((rs2[0].x + rs2[0].y) + (rs2[1].x + rs2[1].y)) +
                                 ((rs2[2].x + rs2[2].y) + (rs2[3].x + rs2[3].y));
                lsum = lsum * alpha + rs;
                if (j > first) {  // PV of the previous tile must be done before O is rescaled
                    ok = pv_done(l - 1);
                    if (!ok) break;
                    pa::tc::fence_after();
                    if (__any_sync(pa::kFull, alpha != 1.f)) {
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            pa::tc::ld32(lane_base + o_col + c0, o);
                            pa::tc::wait_ld();
#pragma unroll
                            for (int c = 0; c < 32; ++c)
                                o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                            pa::tc::st32(lane_base + o_col + c0, o);
                        }
                    }
                }
                // V rows that no row of the item sees may hold anything (slots
                // never written, tokens before the window): P is 0 there, but
                // 0 * NaN is NaN, so they are zeroed.  Each group does so before
                // its own P arrival; both write zeros.
                {
                    const uint32_t vst = skv + ((g0 + j) % NST) * 2 * Lay::T_BYTES + Lay::T_BYTES;
                    auto zero_rows = [&](int a, int b) {
                        for (int idx = row; idx < (b - a) * CH; idx += 128)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                                             vst + pa::tc::sw128(a + idx / CH, idx % CH * 8, kT2KT)),
                                         "r"(0u)
                                         : "memory");
                    };
                    const int past = I.kv_end - j0, ha = max(0, s0), hb = min(kT2KT, I.lo - j0);
                    if (past < kT2KT) zero_rows(past, kT2KT);
                    if (ha < hb) zero_rows(ha, hb);
                    if (past < kT2KT || ha < hb)
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                pa::tc::st32(lane_base + p_col, ph);
                pa::tc::st32(lane_base + p_col + 32, pl);
                pa::tc::wait_st();
                pa::tc::fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[wg]);
            }
            g0 += I.ntiles;
            if (!ok) break;
            const bool any = first < I.ntiles;  // SPLIT: an item of one tile leaves B none
            // (while the last PV runs:) where this lane writes its part of four
            // rows, NULL for rows past the request, and the group's next item
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
            if (any) ok = pv_done(l - 1);       // PV of the item's last tile
            if (!ok) break;
            pa::tc::fence_after();
            // 32 columns of O from column c0, times f
            auto load_o = [&](int c0, float f, float (&o)[32]) {
                uint32_t u[32];
                pa::tc::ld32(lane_base + o_col + c0, u);
                pa::tc::wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = any ? __uint_as_float(u[c]) * f : 0.f;
            };
            // Rounded, through this warp's 2 KB of shared memory, so that four
            // lanes write 64 bytes of a row (a lane writing its own row in
            // 16-byte pieces took 5,000 cycles per item and held up the next
            // item's products)
            uint8_t *stage = smem + Lay::OFF_OUT + warp * 2048;
            auto swz = [](int r, int c) { return r * 64 + ((c ^ ((r >> 1) & 3)) << 4); };
            auto store_o = [&](int c0, const float (&o)[32]) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 w4;
                    w4.x = pack_bf16(o[8 * c], o[8 * c + 1]);
                    w4.y = pack_bf16(o[8 * c + 2], o[8 * c + 3]);
                    w4.z = pack_bf16(o[8 * c + 4], o[8 * c + 5]);
                    w4.w = pack_bf16(o[8 * c + 6], o[8 * c + 7]);
                    *reinterpret_cast<uint4 *>(stage + swz(lane, c)) = w4;
                }
                __syncwarp();
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 w4 = *reinterpret_cast<const uint4 *>(
                        stage + swz(k * 8 + lane / 4, lane & 3));
                    if (dst[k]) *reinterpret_cast<uint4 *>(dst[k] + c0) = w4;
                }
                __syncwarp();
            };
            if constexpr (!SPLIT) {
                const float inv = 1.f / lsum;
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    float o[32];
                    load_o(c0, inv, o);
                    store_o(c0, o);
                }
            } else {
                // Each group finishes half of the columns: it takes the other's
                // part of them and gives its own part of the other half.  B
                // gives first; a row's slots are used by one thread of each.
                float4 *xs = reinterpret_cast<float4 *>(smem + Lay::OFF_X);  // [D / 8][128]
                float2 *xml = reinterpret_cast<float2 *>(smem + Lay::OFF_ML);  // [group][128]
                auto give = [&](int half) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D / 2; c0 += 32) {
                        float o[32];
                        load_o(half * (D / 2) + c0, 1.f, o);
#pragma unroll
                        for (int c = 0; c < 32; c += 4)
                            xs[((c0 + c) / 4) * 128 + row] = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
                    }
                    xml[wg * 128 + row] = make_float2(m_used, lsum);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&x_full[wg]);
                };
                auto take = [&](int half) {
                    if (!__all_sync(pa::kFull, pa::mbar_wait(&x_full[wg ^ 1], it & 1))) return false;
                    const float2 other = xml[(wg ^ 1) * 128 + row];
                    const float M = fmaxf(m_used, other.x);
                    const float fo = other.x == -INFINITY ? 0.f : exp2f(other.x - M);
                    const float fm = m_used == -INFINITY ? 0.f : exp2f(m_used - M);
                    const float inv = 1.f / (lsum * fm + other.y * fo);
#pragma unroll 1
                    for (int c0 = 0; c0 < D / 2; c0 += 32) {
                        float o[32];
                        load_o(half * (D / 2) + c0, fm * inv, o);
#pragma unroll
                        for (int c = 0; c < 32; c += 4) {
                            const float4 v = xs[((c0 + c) / 4) * 128 + row];
                            o[c] = fmaf(v.x, fo * inv, o[c]);
                            o[c + 1] = fmaf(v.y, fo * inv, o[c + 1]);
                            o[c + 2] = fmaf(v.z, fo * inv, o[c + 2]);
                            o[c + 3] = fmaf(v.w, fo * inv, o[c + 3]);
                        }
                        store_o(half * (D / 2) + c0, o);
                    }
                    __syncwarp();
                    return true;
                };
                if (wg == 1) {
                    give(0);
                    ok = take(1);
                } else {
                    ok = take(0);
                    if (ok) give(1);
                }
                ok = __all_sync(pa::kFull, ok);
                if (!ok) break;
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

// Upper bound of the query tiles of qtok tokens: at most one per request is
// partly filled.
int64_t query_tiles(const WinParams &p, int max_query_len, int qtok) {
    return std::min<int64_t>(int64_t(p.R) * ((max_query_len + qtok - 1) / qtok),
                             int64_t(p.T) / qtok + p.R);
}

template <int D, int GQ, bool SPLIT>
int launch_t(const WinParams &p0, const void *q, const void *k_cache, const void *v_cache,
             int max_query_len, int sms, cudaStream_t stream) {
    const int64_t rows = (p0.num_blocks * p0.Hkv) << p0.bs_log2;
    CUtensorMap kmap, vmap, qmap;
    const int box = std::min(p0.bs, kT2KT);
    if (int rc = pa::encode_pool_map(&kmap, k_cache, rows, D, box)) return rc;
    if (int rc = pa::encode_pool_map(&vmap, v_cache, rows, D, box)) return rc;
    if (int rc = pa::encode_q_map(&qmap, q, p0.T, p0.Hq, D, GQ, 128 / GQ)) return rc;
    using Lay = WLayout<D>;
    auto kern = prefill_window_kernel<D, GQ, SPLIT>;
    static std::atomic<uint64_t> attr_done{0};
    if (int rc = set_smem_once(kern, Lay::SMEM, &attr_done)) return rc;
    constexpr int qtok = (SPLIT ? 128 : 256) / GQ;
    // more requests than the kernel's tables hold: several launches
    for (int r0 = 0; r0 < p0.R; r0 += kMaxR) {
        WinParams p = p0;
        p.R = std::min(kMaxR, p0.R - r0);
        p.block_table += int64_t(r0) * p.MB;
        p.query_start += r0;
        p.context_lens += r0;
        const int64_t tiles = query_tiles(p, max_query_len, qtok);
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(
            std::max<int64_t>(1, std::min<int64_t>(sms, tiles * p.Hkv))));
        cfg.blockDim = dim3(Lay::THREADS);
        cfg.dynamicSmemBytes = Lay::SMEM;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
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
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return pa::cuda_fail(cudaGetLastError(), "prefill_window: SM count");
    if (query_tiles(p, max_query_len, 256 / GQ) * p.Hkv * 2 <= sms)
        return launch_t<D, GQ, true>(p, q, k_cache, v_cache, max_query_len, sms, stream);
    return launch_t<D, GQ, false>(p, q, k_cache, v_cache, max_query_len, sms, stream);
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
                                         R, block_size, num_blocks, window, num_sinks, stream))
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
