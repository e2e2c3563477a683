// Linear attention with a decay for each head over chunks of tokens (bf16, tcgen05).
//
// With the state S before a chunk of C = 64 tokens, and i, j its tokens,
//   o_i = scale [ sum_{j <= i} l^(i-j) (q_i . k_j) v_j  +  l^(i+1) q_i S ]
//   S  <- l^C S + sum_j k_j (l^(C-1-j) v_j)^T
// so that a chunk is four products: Q K^T, P V with P = Q K^T times the decays, Q S
// and K^T V'.
//
// Bound: HBM (q, k, v and o: 8 D bytes per token and head) if the products, the
// conversions between them and the copies overlap; a chunk of D = 128 costs 2,800
// cycles of an SM's part of HBM, 1,800 of its tensor core and 2,400 issue
// slots of each scheduler.  Hence one CTA per (request, head) with a warp group for each job:
//   warps 0-3, 4-7  the state, in registers in fp32 (thread = value dimension, half of
//                   the key dimensions each): adds a chunk's K^T V' to it and gives
//                   it to the next chunk's Q S as two bf16 terms in TMEM; in between
//                   0, 1, 4, 5 (and 13) write P as two bf16 terms to shared memory, and
//                   7 has the chunk after the ring's copied in
//   warp 9          issues the tcgen05.mma
//   warps 8, 10, 11 V' = l^(C-1-j) v_j as three bf16 terms in shared memory, 32 tokens at
//                   a time (the other 32 are in use meanwhile).  P is made by warps of
//                   schedulers 0 and 1, so 8 has a smaller share than 10 and 11
//   warps 12-15     outputs; without outputs 13 has a quarter of V', and 15 copies
// Outputs are computed transposed (lanes = value dimensions, columns = tokens), so the
// state is an operand that lies in TMEM, where the threads that own it write it;
// with tokens as lanes it would take 64 KB of shared memory.  Q K^T has its tokens
// in lanes 0-63; the other lanes, and for D = 64 the value dimensions from 64 on,
// hold products of whatever lies behind the operand and are never read.
//
// Terms: a state's own sums (K^T V') take V' in three bf16 terms, as exact as its
// fp32 accumulation; P and S enter an output, which is rounded to bf16, in two
// (2^-16 of a term).
//
// Few (request, head) pairs leave SMs idle: then a request's tokens are cut into
// segments.  One launch sums each segment's own state (the kernel without its output
// part), one chains them, and the segments then run like requests.
//
// Measured (32 heads, D 128): 8 requests of 65 to 2,048 tokens 73 us, 3.9 TB/s (0.57 of
// HBM); a prompt of 16,384 tokens, 4 segments, 214 us call after call (70 of them the
// segments' sums; 219 with an L2 that holds nothing of it, and 529 uncut); 100 tokens 9.5 us.  A chunk takes about 4,000 cycles: the sequence of
// waits, issues and commits of warp 9 (each 150 to 400 cycles, with what 16 warps of five
// roles lose to instruction fetches), beside 2,900 of V' and 2,700 of the state's warps;
// the tensor core is busy for 38 % of the time, issue 55 %.  Shared memory has 2,800 cycles
// of it to move, at 128 bytes each: 48 KB copied in, 224 KB of operands (96 of K^T V', whose
// three terms read K three times), 64 KB for V', 16 for P; without outputs 1,500 of 2,100,
// and more warps for V' gain nothing there (220 us for the prompt with six).
#include <algorithm>
#include <climits>
#include <cmath>

#include "pa_linear.cuh"

namespace {

using namespace pa::pf;
using pa::lin::LinParams;
using pa::lin::Request;

constexpr int C = 64;  // tokens per chunk
constexpr int kSortedR = 64;  // requests that a CTA puts in order

struct ChunkParams {
    LinParams p;
    float *ws;     // [slots][H][D][D]: segments' sums, then the states before them
    int seg;       // tokens per segment (a multiple of C); 0: whole requests
    int slots;     // segments that the grid and the workspace have room for
    bool sorted;   // whole requests, more CTAs than SMs: long ones first
};

template <int D>
struct Lay {
    static constexpr int THREADS = 16 * 32;  // 128 registers each
    static constexpr int MMA_WARP = 9, P_WARP = 13;
    static constexpr int NST = D == 128 ? 3 : 4;
    static constexpr int TILE = C * D * 2;       // a chunk's q, k or v
    static constexpr int STAGE = 3 * TILE;       // q, k, v
    static constexpr int OFF_VP = NST * STAGE;   // V' terms
    static constexpr int P_TERM = C * C * 2;
    static constexpr int OFF_P = OFF_VP + 3 * TILE;  // [buffer][term]
    static constexpr int OFF_BAR = OFF_P + 4 * P_TERM;
    // full, empty [NST]; s1_full, p_full, vp_full [2]; u_half, u_full, u_free, s_full,
    // o_done, o_free, drain
    static constexpr int N_BAR = 2 * NST + 6 + 7;
    static constexpr int OFF_F = (OFF_BAR + N_BAR * 8 + 15) / 16 * 16;  // scale l^(i+1)
    static constexpr int OFF_W = OFF_F + C * 4;        // l^(C-1-j), and of the last chunk
    static constexpr int OFF_D = OFF_W + 2 * C * 4;    // l^x, x = 1 - C .. C - 1 (1 below 0)
    static constexpr int OFF_MISC = OFF_D + 2 * C * 4; // TMEM slot, fail flag
    static constexpr int OFF_L = OFF_MISC + 16;        // l^C, l^(tokens of the last chunk)
    static constexpr int SMEM = OFF_L + 16 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory");
    static_assert(OFF_VP % 1024 == 0 && OFF_P % 1024 == 0 && OFF_BAR % 8 == 0 && OFF_F % 16 == 0 && OFF_MISC % 8 == 0,
                  "alignment");
    static constexpr int TMEM_COLS = 512;
    static constexpr int U = 0, S = D, S1 = 2 * D, O2 = S1 + 2 * C, O1 = O2 + C;
    static_assert(O1 + C <= TMEM_COLS, "tensor memory");
    static constexpr int LANE_WARPS = D / 32;  // warps of a group whose lanes mean something
};

// A CTA's work: tokens [t0, t0 + n) of head h; the state before them and where the
// state behind them goes (NULL: nothing, nowhere).
struct Work {
    int t0, n, h;
    const float *from;
    float *to;
};

// Segments of a request.
__device__ __forceinline__ int segments(const ChunkParams &a, const Request &x) {
    return x.state < 0 ? 0 : a.seg ? (x.n + a.seg - 1) / a.seg : 1;
}

// The request that owns segment `slot`, and the slot of its first one; false if none
// does.  Whole warp, the same for all.
__device__ __forceinline__ bool find_request(const ChunkParams &a, int slot, int *r, int *first) {
    const int lane = threadIdx.x & 31;
    int carry = 0;
    for (int r0 = 0; r0 < a.p.R; r0 += 32) {
        const int ns = r0 + lane < a.p.R ? segments(a, pa::lin::request(a.p, r0 + lane)) : 0;
        int incl = ns;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(pa::kFull, incl, o);
            if (lane >= o) incl += y;
        }
        const int f = carry + incl - ns;
        const unsigned mine = __ballot_sync(pa::kFull, slot >= f && slot < f + ns && f + ns <= a.slots);
        if (mine) {
            const int src = __ffs(mine) - 1;
            *r = r0 + src;
            *first = __shfl_sync(pa::kFull, f, src);
            return true;
        }
        carry += __shfl_sync(pa::kFull, incl, 31);
    }
    return false;
}

// The slot-th request in the order of the tokens' number, most first.  Whole CTA of 512
// threads, 8 for each request; `table`: kSortedR + 1 words that nobody uses yet.
__device__ __forceinline__ int in_order(const ChunkParams &a, int slot, int *table) {
    const int i = threadIdx.x >> 3, part = threadIdx.x & 7;
    const int n = i < a.p.R ? a.p.query_start[i + 1] - a.p.query_start[i] : INT_MIN;
    if (part == 0) table[i] = n;
    __syncthreads();
    int rank = 0;
#pragma unroll
    for (int k = 0; k < kSortedR / 8; ++k) {
        const int y = k * 8 + part, m = table[y];
        rank += m > n || (m == n && y < i);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(pa::kFull, rank, o);
    if (part == 0 && rank == slot) table[kSortedR] = i;
    __syncthreads();
    return table[kSortedR];
}

template <int D, bool SUM>
__device__ __forceinline__ Work find_work(const ChunkParams &a, int *table) {
    Work w{0, 0, 0, nullptr, nullptr};
    const int slot = blockIdx.x / a.p.H;
    w.h = blockIdx.x % a.p.H;
    int r = !SUM && a.sorted ? in_order(a, slot, table) : slot, first = 0;
    if (a.seg && !find_request(a, slot, &r, &first)) return w;
    const Request x = pa::lin::request(a.p, r);
    if (x.state < 0) return w;
    constexpr int64_t DD = D * D;
    float *pool = a.p.states + (static_cast<int64_t>(x.state) * a.p.H + w.h) * DD;
    float *own = a.ws + (static_cast<int64_t>(slot) * a.p.H + w.h) * DD;
    if (!a.seg) {
        w.t0 = x.t0;
        w.n = x.n;
        w.from = x.held ? pool : nullptr;
        w.to = pool;
        return w;
    }
    const int s = slot - first;
    const bool last = s == segments(a, x) - 1;
    if (SUM && last) return w;  // (the state behind the last segment comes from its own run)
    w.t0 = x.t0 + s * a.seg;
    w.n = min(a.seg, x.n - s * a.seg);
    w.from = SUM ? nullptr : own;
    w.to = SUM ? own : last ? pool : nullptr;
    return w;
}

// The chunk of tokens t0 .. of head h into shared memory, completing on `bar`.
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap *map, int h, int t0, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %2}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(h), "r"(t0), "r"(pa::smem_u32(bar))
        : "memory");
}
// x as two or three bf16 terms, two values at a time: a term that is not the last, and
// what it leaves.  It stays finite: an infinity, or a number past bf16's range, is left to
// the last term, where inf - inf would be NaN.
__device__ __forceinline__ uint32_t take_bf16(float2 &x) {
    uint32_t t;
    asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(t) : "f"(x.y), "f"(x.x));
    x = pa::ffma2(pa::bf16x2_to_float2(t), make_float2(-1.f, -1.f), x);
    return t;
}

template <int D, bool SUM>
__global__ void __launch_bounds__(Lay<D>::THREADS, 1)
    chunk_kernel(const ChunkParams a, const __grid_constant__ CUtensorMap qmap,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using L = Lay<D>;
    constexpr int NST = L::NST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = pa::smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + L::OFF_BAR);
    uint64_t *full = bars, *empty = full + NST, *s1_full = empty + NST,
             *p_full = s1_full + 2, *vp_full = p_full + 2, *u_half = vp_full + 2, *u_full = u_half + 1, *u_free = u_full + 1,
             *s_full = u_free + 1, *o_done = s_full + 1, *o_free = o_done + 1,
             *drain = o_free + 1;
    float *fdec = reinterpret_cast<float *>(smem + L::OFF_F), *wdec = reinterpret_cast<float *>(smem + L::OFF_W),
          *pdec = reinterpret_cast<float *>(smem + L::OFF_D) + C;
    pa::lin::Decay *chunk_decay = reinterpret_cast<pa::lin::Decay *>(smem + L::OFF_L);
    // Without outputs K^T V' has two places, so that the tensor core goes on while the state
    // takes one: the scores' barriers, which are free then, say full and taken.
    uint64_t *sum_full = s1_full, *sum_free = p_full;
    auto u_col = [](int c) { return L::U + (SUM ? (c & 1) * D : 0); };
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + L::OFF_MISC);
    volatile int *fail = reinterpret_cast<volatile int *>(smem + L::OFF_MISC + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // ---- set-up: barriers, TMEM ------------------------------------------------
    if (tid == 0) {
        for (const CUtensorMap *map : {&qmap, &kmap, &vmap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
        for (int i = 0; i < NST; ++i) {
            pa::mbar_init(&full[i], 1);
            pa::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            pa::mbar_init(&s1_full[i], 1);
            pa::mbar_init(&p_full[i], SUM ? 2 * L::LANE_WARPS : 5);
            pa::mbar_init(&vp_full[i], SUM ? 4 : 3);
        }
        pa::mbar_init(u_half, 1);
        pa::mbar_init(u_full, 1);
        pa::mbar_init(u_free, 2 * L::LANE_WARPS);
        pa::mbar_init(s_full, 2 * L::LANE_WARPS);
        pa::mbar_init(o_done, 1);
        pa::mbar_init(o_free, L::LANE_WARPS);
        pa::mbar_init(drain, 1);
        *fail = 0;
        pa::fence_barrier_init();
    }
    if (warp == L::MMA_WARP) pa::tc::alloc(tslot, L::TMEM_COLS);
    // P of the first 32 tokens and the last 32: always 0 (both buffers and terms)
    for (int x = tid; x < 4 * 32 * 4; x += L::THREADS) {
        const int i = x >> 2 & 31;
        *reinterpret_cast<uint4 *>(smem + L::OFF_P + (x >> 7) * L::P_TERM + i * 128 + (((x & 3) + 4) ^ (i & 7)) * 16) =
            make_uint4(0, 0, 0, 0);
    }
    pa::fence_proxy_async();
    // launched as a programmatic dependent: the inputs are ready past this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Work w = find_work<D, SUM>(a, reinterpret_cast<int *>(smem + L::OFF_VP));
    const float g = pa::lin::log_decay(a.p, w.h);
    const int nc = (w.n + C - 1) / C, rest = w.n - (nc - 1) * C;  // chunks, tokens of the last
    {  // a power for each of 4 C threads
        const int i = tid % C, what = tid / C;
        if (what < 4) {
            const int n = what == 0 ? i + 1 : what == 1 ? C - 1 - i : what == 2 ? i : max(rest - 1 - i, 0);
            const float x = pa::lin::decay_power(g, n);
            if (what == 0) fdec[i] = a.p.scale * x;
            else if (what == 1) wdec[i] = x;
            else if (what == 2) pdec[i] = x;
            else wdec[C + i] = i < rest ? x : 0.f;
        } else if (what == 4) {
            pdec[i - C] = 1.f;
        } else if (what == 5 && i < 2) {
            chunk_decay[i] = pa::lin::decay_factor(g, i ? rest : C);
        }
    }
    pa::tc::fence_before();
    __syncthreads();
    pa::tc::fence_after();
    const uint32_t tmem = *tslot;
    int loads_issued = 0;
    auto signal = [&](uint64_t *bar) {  // one arrival per warp, behind its writes
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    constexpr int LOAD_WARP = SUM ? 15 : 7;
    // Copies of chunk c into its stage (that warp).  Whole tiles of 64 tokens: rows past the
    // work's tokens are other tokens' (or zeros past the last), see below.
    auto load = [&](int c) {
        constexpr int FIRST = SUM ? 1 : 0;  // (no q)
        const int st = c % NST;
        if (lane == 0) {
            pa::mbar_arrive_expect_tx(&full[st], (3 - FIRST) * L::TILE);
            ++loads_issued;
#pragma unroll
            for (int x = FIRST; x < 3; ++x)
                load_rows(s0 + st * L::STAGE + x * L::TILE, x == 0 ? &qmap : x == 1 ? &kmap : &vmap, w.h, w.t0 + c * C,
                          &full[st]);
        }
        __syncwarp();
    };
    // The loads behind the ring's first, by a warp that does nothing else.
    auto load_all = [&]() {
        for (int c = NST; c < nc; ++c) {
            if (!wait_all(&empty[c % NST], ((c / NST) - 1) & 1)) {
                *fail = 1;
                break;
            }
            load(c);
        }
    };
    if (warp == LOAD_WARP)
        for (int c = 0; c < min(nc, NST); ++c) load(c);

    // P of chunk c, columns j0 .. j1 (whole 16s): lane = token i of the chunk (warps whose
    // lanes are 0-63).  Of tokens 0-31 the columns from 32 on are 0 and stay so.
    auto make_p = [&](int c, int j0, int j1) {
        const int row = (warp & 1) * 32 + lane;
        const uint32_t from = tmem + (static_cast<uint32_t>((warp & 1) * 32) << 16) + L::S1 + (c & 1) * C;
        if (!wait_all(&s1_full[c & 1], (c >> 1) & 1)) return false;
        pa::tc::fence_after();
        const uint32_t to = s0 + L::OFF_P + (c & 1) * 2 * L::P_TERM + row * 128;
#pragma unroll 1
        for (; j0 < j1; j0 += 16) {
            uint32_t hi[8], lo[8], u[16];
            pa::tc::ld16(from + j0, u);
            const float *f = pdec + (row - j0);  // l^(row - j): neighbours in neighbouring lanes
            float2 x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = make_float2(f[-2 * e], f[-2 * e - 1]);
            pa::tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (a score of a later token may be anything, also NaN)
                x[e].x = j0 + 2 * e <= row ? x[e].x * __uint_as_float(u[2 * e]) : 0.f;
                x[e].y = j0 + 2 * e < row ? x[e].y * __uint_as_float(u[2 * e + 1]) : 0.f;
                hi[e] = take_bf16(x[e]);
                lo[e] = pack_bf16(x[e].x, x[e].y);
            }
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const uint32_t at = to + ((((j0 + 2 * e) >> 3) ^ (row & 7)) << 4);
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(hi[e]), "r"(hi[e + 1]),
                             "r"(hi[e + 2]), "r"(hi[e + 3])
                             : "memory");
                asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + L::P_TERM), "r"(lo[e]),
                             "r"(lo[e + 1]), "r"(lo[e + 2]), "r"(lo[e + 3])
                             : "memory");
            }
        }
        pa::tc::fence_before();
        pa::fence_proxy_async();
        signal(&p_full[c & 1]);
        return true;
    };

    if (warp == L::MMA_WARP) {
        // ---------------- MMA ----------------
        constexpr uint32_t kIdS1 = pa::tc::idesc_bf16(128, C, 0, 0);  // Q K^T
        constexpr uint32_t kIdU = pa::tc::idesc_bf16(128, D, 1, 1);   // V'^T K
        constexpr uint32_t kIdO1 = pa::tc::idesc_bf16(128, C, 1, 0);  // V^T P^T
        constexpr uint32_t kIdO2 = pa::tc::idesc_bf16(128, C, 0, 0);  // S^T Q^T
        constexpr uint32_t kStage = L::STAGE >> 4, kTile = L::TILE >> 4;
        // rows of 128 bytes, K-major; tokens as K (64 tokens per column block)
        const uint64_t row_major = pa::tc::sdesc(s0, 16, 1024), col_major = pa::tc::sdesc(s0, C * 128, 1024);
        // The whole warp goes along and one lane issues: descriptors and waits stay uniform
        // (one lane alone took 294 us for a prompt of 16,384 tokens, then 219 with all).  S1
        // of a chunk is overwritten two chunks later, its P has been waited for by then.
        auto issue_s1 = [&](int c) {
            if (!wait_all(&full[c % NST], (c / NST) & 1)) return false;
            pa::tc::fence_after();
            if (pa::tc::elect_one()) {
                const uint64_t q = row_major + static_cast<uint32_t>((c % NST) * kStage), k = q + kTile;
#pragma unroll 1
                for (int b = 0; b < D / 64; ++b)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint32_t off = (b * C * 128 + ks * 32) >> 4;
                        pa::tc::mma_ss(tmem + L::S1 + (c & 1) * C, q + off, k + off, kIdS1, b + ks > 0);
                    }
                pa::tc::commit(&s1_full[c & 1]);
            }
            __syncwarp();
            return true;
        };
        bool ok = SUM || nc == 0 || issue_s1(0);
        for (int c = 0; c < nc && ok; ++c) {
            const uint32_t stage = static_cast<uint32_t>((c % NST) * kStage);
            if (SUM) ok = wait_all(&full[c % NST], (c / NST) & 1);
            // the state has what lies in the place of this K^T V'
            if (SUM && c > 1) ok = ok && wait_all(&sum_free[c & 1], ((c >> 1) - 1) & 1);
            if (!SUM && c > 0) ok = ok && wait_all(u_free, (c - 1) & 1);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                ok = ok && wait_all(&vp_full[half], c & 1);
                if (!ok) break;
                pa::tc::fence_after();
                if (pa::tc::elect_one()) {
                    const uint64_t k = col_major + stage + kTile, vp = col_major + (L::OFF_VP >> 4);
#pragma unroll 1
                    for (int ks = half * C / 32; ks < (half + 1) * C / 32; ++ks)
#pragma unroll
                        for (int term = 0; term < 3; ++term)
                            pa::tc::mma_ss(tmem + u_col(c), vp + term * kTile + ((ks * 16 * 128) >> 4),
                                           k + ((ks * 16 * 128) >> 4), kIdU, ks + term > 0);
                    pa::tc::commit(half ? u_full : u_half);
                    if (SUM && half) {
                        pa::tc::commit(&sum_full[c & 1]);
                        pa::tc::commit(&empty[c % NST]);
                    }
                }
                __syncwarp();
            }
            if (!ok) break;
            if (SUM) continue;
            if (c + 1 < nc) ok = issue_s1(c + 1);
            ok = ok && wait_all(&p_full[c & 1], (c >> 1) & 1) && (c == 0 || wait_all(o_free, (c - 1) & 1));
            if (!ok) break;
            pa::tc::fence_after();
            if (pa::tc::elect_one()) {
                const uint64_t v = col_major + stage + 2 * kTile;
                const uint64_t p = row_major + ((L::OFF_P + (c & 1) * 2 * L::P_TERM) >> 4);
#pragma unroll 1
                for (int ks = 0; ks < C / 16; ++ks)
#pragma unroll
                    for (int term = 0; term < 2; ++term)
                        pa::tc::mma_ss(tmem + L::O1, v + ((ks * 16 * 128) >> 4),
                                       p + ((term * L::P_TERM + ks * 32) >> 4), kIdO1, ks + term > 0);
            }
            __syncwarp();
            ok = wait_all(s_full, c & 1);
            if (!ok) break;
            pa::tc::fence_after();
            if (pa::tc::elect_one()) {
                const uint64_t q = row_major + stage;
#pragma unroll 1
                for (int b = 0; b < D / 64; ++b)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                        for (int term = 0; term < 2; ++term)
                            pa::tc::mma_ts(tmem + L::O2, tmem + L::S + term * (D / 2) + b * 32 + ks * 8,
                                           q + ((b * C * 128 + ks * 32) >> 4), kIdO2, b + ks + term > 0);
                pa::tc::commit(o_done);  // (of O1 too: every product issued before)
                if (D == 64) pa::tc::commit(&empty[c % NST]);
            }
            __syncwarp();
        }
        if (!ok) *fail = 1;
    } else if (warp < 8) {
        // ---------------- the state ----------------
        constexpr int HALF = D / 2;  // key dimensions of this warp group
        const int k0 = warp < 4 ? 0 : HALF, dv = (warp & 3) * 32 + lane;
        const uint32_t base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        if (dv < D) {
            float2 s[HALF / 2];
#pragma unroll
            for (int k = 0; k < HALF; k += 2)
                s[k / 2] = w.from ? make_float2(w.from[(k0 + k) * D + dv], w.from[(k0 + k + 1) * D + dv])
                                  : make_float2(0.f, 0.f);
            auto give = [&]() {  // to the next Q S
#pragma unroll
                for (int k = 0; k < HALF / 2; k += 8) {
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        // (not before the wait ahead of this: state and terms together
                        // are more than a thread's registers)
                        asm volatile("" : "+f"(s[k + e].x), "+f"(s[k + e].y));
                        float2 x = s[k + e];
                        hi[e] = take_bf16(x);
                        lo[e] = pack_bf16(x.x, x.y);
                    }
                    pa::tc::st8(base + L::S + k0 / 2 + k, hi);
                    pa::tc::st8(base + L::S + (D + k0) / 2 + k, lo);
                }
                pa::tc::wait_st();
                pa::tc::fence_before();
                signal(s_full);
            };
            // P: warps 0 and 4 have tokens 0-31, 1 and 5 (and 13) tokens 32-63
            const bool has_p = (warp & 3) < 2;
            const int j0 = (warp >> 2) * 16;
            bool ok = true;
            if (!SUM && nc > 0) {
                give();
                if (has_p) ok = make_p(0, j0, j0 + 16);
            }
            for (int c = 0; c < nc && ok; ++c) {
                const pa::lin::Decay l = chunk_decay[c + 1 == nc];  // (kept there: registers are short)
                const float2 hi = make_float2(l.hi, l.hi), lo = make_float2(l.lo, l.lo);
                ok = SUM ? wait_all(&sum_full[c & 1], (c >> 1) & 1) : wait_all(u_full, c & 1);
                if (!ok) break;
                pa::tc::fence_after();
#pragma unroll
                for (int k = 0; k < HALF / 2; k += 8) {
                    uint32_t u[16];
                    pa::tc::ld16(base + u_col(c) + k0 + 2 * k, u);
                    pa::tc::wait_ld();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[k + e] = pa::ffma2(hi, s[k + e],
                                             pa::ffma2(lo, s[k + e], make_float2(__uint_as_float(u[2 * e]),
                                                                                 __uint_as_float(u[2 * e + 1]))));
                }
                pa::tc::fence_before();
                signal(SUM ? &sum_free[c & 1] : u_free);
                if (!SUM && c + 1 < nc) {
                    // (the place of this P was read before the last Q S)
                    if (has_p) ok = make_p(c + 1, j0, j0 + 16);
                    ok = ok && wait_all(o_done, c & 1);  // the last Q S has read its state
                    if (!ok) break;
                    pa::tc::fence_after();
                    if (warp == LOAD_WARP && c + NST < nc) load(c + NST);
                    give();
                }
            }
            if (!ok) *fail = 1;
            else if (w.to && nc > 0) {
#pragma unroll
                for (int k = 0; k < HALF; k += 2) {
                    w.to[(k0 + k) * D + dv] = s[k / 2].x;
                    w.to[(k0 + k + 1) * D + dv] = s[k / 2].y;
                }
            }
        } else if (!SUM && warp == LOAD_WARP) {  // (D = 64)
            load_all();
        }
    } else if (warp < 12 || (SUM && warp == 13)) {
        // ---------------- V' ----------------
        // 16 bytes at a time, at the same place of the tile: whatever the swizzle, byte
        // x of a column block belongs to token x / 128.  Four loads at once, as each
        // takes longer than the work on it.
        constexpr int PIECES = C * D / 16;  // of half the tokens
        constexpr int MOST = PIECES / 32 * (SUM ? 4 : 6) / 16;  // per thread: 4 of 16 parts each, or 4, 6 and 6
        const int part = SUM ? (warp == 13 ? 12 : (warp - 8 - (warp > 8)) * 4) : warp == 8 ? 0 : warp == 10 ? 4 : 10;
        const int mine = SUM || warp > 8 ? MOST : PIECES / 32 * 4 / 16, first = PIECES / 16 * part + lane;
        constexpr int NB = SUM && D == 128 ? 4 : 2;
        // byte offset of a thread's k-th piece
        auto place = [&](int half, int k) {
            const int y = first + k * 32;
            return ((y >> 8) * 512 + half * 256 + (y & 255)) * 16;
        };
        bool ok = true;
        for (int c = 0; c < nc && ok; ++c) {
            const int m = c + 1 < nc ? C : rest;
            const float *wt = wdec + (c + 1 < nc ? 0 : C);
            ok = wait_all(&full[c % NST], (c / NST) & 1);
            if (!ok) break;
            const uint32_t kt = s0 + (c % NST) * L::STAGE + L::TILE, vt = kt + L::TILE;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (m < C) {
                    // no tokens of this work: their V and K may hold anything, and 0 x NaN is NaN
                    for (int k = 0; k < mine; ++k) {
                        const int x = place(half, k);
                        if (((x >> 7) & (C - 1)) >= m)
                            for (const uint32_t at : {kt + x, vt + x})
                                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(at), "r"(0u) : "memory");
                    }
                    __syncwarp();  // (a lane reads back what it wrote)
                }
                // NB pieces at once, the next on their way (the last of an odd number twice).
                uint4 v[NB];
                float f[NB];
                auto fetch = [&](int k0) {
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const int x = place(half, min(k0 + k, mine - 1));
                        v[k] = pa::lds128(vt + x);
                        f[k] = wt[(x >> 7) & (C - 1)];
                    }
                };
                fetch(0);
                if (c > 0) ok = wait_all(half ? u_full : u_half, (c - 1) & 1);
                if (!ok) break;
                // (not unrolled further: the roles' loops together have to stay near the
                // instruction caches)
#pragma unroll 1
                for (int k0 = 0; k0 < mine; k0 += NB) {
                    float2 y[NB][4];
                    uint32_t t[NB][3][4];
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        pa::Elem<__nv_bfloat16>::unpack(v[k], y[k]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[k][e] = __fmul2_rn(y[k][e], make_float2(f[k], f[k]));
                    }
                    fetch(k0 + NB);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int k = 0; k < NB; ++k) {
                            t[k][0][e] = take_bf16(y[k][e]);
                            t[k][1][e] = take_bf16(y[k][e]);
                            t[k][2][e] = pack_bf16(y[k][e].x, y[k][e].y);
                        }
#pragma unroll
                    for (int k = 0; k < NB; ++k) {
                        const uint32_t at = s0 + L::OFF_VP + place(half, min(k0 + k, mine - 1));
#pragma unroll
                        for (int term = 0; term < 3; ++term)
                            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at + term * L::TILE),
                                         "r"(t[k][term][0]), "r"(t[k][term][1]), "r"(t[k][term][2]),
                                         "r"(t[k][term][3])
                                         : "memory");
                    }
                }
                pa::fence_proxy_async();
                signal(&vp_full[half]);
            }
        }
        if (!ok) *fail = 1;
    } else if (SUM) {
        if (warp == LOAD_WARP) load_all();  // (12 and 14 are idle)
    } else if (warp < 12 + L::LANE_WARPS) {
        // ---------------- outputs ----------------
        const int lw = warp & 3, row = lw * 32 + lane;
        const uint32_t base = tmem + (static_cast<uint32_t>(lw * 32) << 16);
        const int64_t step = static_cast<int64_t>(a.p.H) * D;
        bool ok = true;
        auto put_o = [&](int c) {  // row = value dimension
            if (!wait_all(o_done, c & 1)) return false;
            pa::tc::fence_after();
            // Lanes 2 x and 2 x + 1 trade: the even one writes both dimensions of token i,
            // the odd one of token i + 4, 16 lanes 64 bytes.
            const bool odd = lane & 1;
            const int m = (c + 1 < nc ? C : rest) - (odd ? 4 : 0);
            __nv_bfloat16 *to = static_cast<__nv_bfloat16 *>(a.p.out) +
                                (static_cast<int64_t>(w.t0 + c * C + (odd ? 4 : 0)) * a.p.H + w.h) * D + (row & ~1);
#pragma unroll 1
            for (int i0 = 0; i0 < C; i0 += 16) {
                uint32_t x1[16], x2[16];
                pa::tc::ld16(base + L::O1 + i0, x1);
                pa::tc::ld16(base + L::O2 + i0, x2);
                float o[16], got[8];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(fdec + i0 + e);
                    o[e] = f.x, o[e + 1] = f.y, o[e + 2] = f.z, o[e + 3] = f.w;
                }
                pa::tc::wait_ld();
                if (i0 + 16 == C) {
                    pa::tc::fence_before();
                    signal(o_free);
                }
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    o[e] = fmaf(o[e], __uint_as_float(x2[e]), a.p.scale * __uint_as_float(x1[e]));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = (e & 3) + 8 * (e >> 2);  // tokens i and i + 4
                    got[e] = __shfl_xor_sync(pa::kFull, odd ? o[i] : o[i + 4], 1);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = (e & 3) + 8 * (e >> 2);
                    const uint32_t v = odd ? pack_bf16(got[e], o[i + 4]) : pack_bf16(o[i], got[e]);
                    if (i0 + i < m) *reinterpret_cast<uint32_t *>(to + (i0 + i) * step) = v;
                }
            }
            return true;
        };
        // (P of tokens 32-63, columns 32-63)
        if (nc > 0 && warp == L::P_WARP) ok = make_p(0, 32, 64);
        for (int c = 0; c < nc && ok; ++c) {
            if (c + 1 < nc && warp == L::P_WARP) ok = make_p(c + 1, 32, 64);
            ok = ok && put_o(c);
        }
        if (!ok) *fail = 1;
    }

    // ---- tear-down ----------------------------------------------------------------
    pa::tc::fence_before();
    __syncthreads();
    if (*fail) {
        // a wait ran out: record it, then let the MMAs and the copies in flight land
        // (bounded) before TMEM and shared memory go away
        if (tid == 0) pa::record_error(a.p.err, PA_DEVERR_TIMEOUT);
        if (warp == L::MMA_WARP) {
            if (pa::tc::elect_one()) pa::tc::commit(drain);
            __syncwarp();
            (void)pa::mbar_wait(drain, 0);
        }
        if (warp == LOAD_WARP && lane == 0)
            for (int st = 0; st < NST && st < loads_issued; ++st)  // the last into each stage
                (void)pa::mbar_wait(&full[st], (loads_issued - 1 - st) / NST & 1);
        pa::tc::fence_before();
        __syncthreads();
    }
    if (warp == L::MMA_WARP) {
        pa::tc::fence_after();
        pa::tc::dealloc(tmem, L::TMEM_COLS);
    }
}

// The states before each segment from the segments' own sums, four elements of one
// (request, head) per thread; `ws` holds the former afterwards.
template <int D>
__global__ void __launch_bounds__(256) chain_kernel(const ChunkParams a) {
    constexpr int PER = D * D / 4 / 256;  // CTAs per (request, head)
    const int x = blockIdx.x / PER, r = x / a.p.H, h = x % a.p.H;
    const int e = (blockIdx.x % PER) * 256 + threadIdx.x;  // of 16 bytes
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Request q = pa::lin::request(a.p, r);
    // the segments of the requests before this one
    __shared__ int before;
    if (threadIdx.x == 0) before = 0;
    __syncthreads();
    int mine = 0;
    for (int i = threadIdx.x; i < r; i += 256) mine += segments(a, pa::lin::request(a.p, i));
    if (mine) atomicAdd(&before, mine);
    __syncthreads();
    const int ns = segments(a, q);
    if (ns == 0) return;
    if (before + ns > a.slots) {  // (the requests' rows overlap: the others run)
        if (threadIdx.x == 0) pa::record_error(a.p.err, PA_DEVERR_BAD_REQUEST);
        return;
    }
    constexpr int64_t DD4 = D * D / 4;
    const pa::lin::Decay l = pa::lin::decay_factor(pa::lin::log_decay(a.p, h), a.seg);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (q.held) s = reinterpret_cast<const float4 *>(a.p.states)[(static_cast<int64_t>(q.state) * a.p.H + h) * DD4 + e];
    float4 *at = reinterpret_cast<float4 *>(a.ws) + (static_cast<int64_t>(before) * a.p.H + h) * DD4 + e;
    const int64_t step = a.p.H * DD4;
    constexpr int AHEAD = 4;  // sums requested before they are needed
    for (int i0 = 0; i0 < ns; i0 += AHEAD) {
        float4 u[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i0 + k < ns - 1) u[k] = at[(i0 + k) * step];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            if (i0 + k >= ns) break;
            at[(i0 + k) * step] = s;
            if (i0 + k == ns - 1) break;
            s.x = pa::lin::decayed(l, s.x, u[k].x);
            s.y = pa::lin::decayed(l, s.y, u[k].y);
            s.z = pa::lin::decayed(l, s.z, u[k].z);
            s.w = pa::lin::decayed(l, s.w, u[k].w);
        }
    }
}

template <typename K, typename... Args>
int go(K kern, int64_t ctas, int threads, size_t smem, cudaStream_t stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    (void)cudaGetLastError();  // drop a stale error that is not ours
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    if (e != cudaSuccess) return pa::cuda_fail(e, "linear_prefill launch");
    return pa::check_launch("linear_prefill launch");
}

template <int D>
int launch(const ChunkParams &a, cudaStream_t stream) {
    using L = Lay<D>;
    static std::atomic<uint64_t> done{0}, done_sum{0};
    if (int rc = set_smem_once(chunk_kernel<D, false>, L::SMEM, &done)) return rc;
    if (int rc = set_smem_once(chunk_kernel<D, true>, L::SMEM, &done_sum)) return rc;
    CUtensorMap q, k, v;
    if (int rc = pa::encode_rows_map(&q, a.p.q, a.p.T, a.p.q_stride, a.p.H, D, C)) return rc;
    if (int rc = pa::encode_rows_map(&k, a.p.k, a.p.T, a.p.k_stride, a.p.H, D, C)) return rc;
    if (int rc = pa::encode_rows_map(&v, a.p.v, a.p.T, a.p.v_stride, a.p.H, D, C)) return rc;
    const int64_t ctas = int64_t(a.seg ? a.slots : a.p.R) * a.p.H;
    if (a.seg) {
        if (int rc = go(chunk_kernel<D, true>, ctas, L::THREADS, L::SMEM, stream, a, q, k, v)) return rc;
        if (int rc = go(chain_kernel<D>, int64_t(a.p.R) * a.p.H * (D * D / 4 / 256), 256, 0, stream, a)) return rc;
    }
    return go(chunk_kernel<D, false>, ctas, L::THREADS, L::SMEM, stream, a, q, k, v);
}

}  // namespace

namespace pa {
namespace lin {

Segments segments_for(int R, int T, int max_query_len, int H) {
    Segments s{0, 0};
    // In chunks: a CTA costs about OVERHEAD besides its own (set-up, state in and out),
    // the launch that sums the segments SUM of one that does it all, and the launches
    // between them LAUNCHES.  Waves are counted as if the tokens were spread evenly; the
    // longest request sets how many chunks follow one another.  Of 15 batches (1 to 32
    // heads, 400 to 16,000 tokens, 1 to 4 requests) the choice was the fastest of up to ten
    // cuts in ten, within 20 % of it in four, and 162 against 122 us for one request of
    // 8,000 tokens among short ones (137 and 123 beside one of 500).  L2 flushed, 32 heads: a
    // prompt of 16,384 tokens 529 us in 1 piece, 284 in 3, 219 in 4 (chosen), 280 in 5, 238 in
    // 8, 223 in 9, 237 in 14, 275 in 16; two of 4,000 tokens 140 in 1 (chosen), 124 in 2.
    constexpr double OVERHEAD = 8, SUM = 0.6, LAUNCHES = 6;
    const int64_t pairs = int64_t(R) * H, most = (int64_t(std::min(max_query_len, T)) + C - 1) / C;
    const int sms = sm_count();
    const double all = (double(T) / C + 0.5 * R) * H / sms;  // chunks per SM
    auto waves = [&](double ctas) { return std::ceil(ctas / sms); };
    double best = std::max(double(most + OVERHEAD), all + waves(double(pairs)) * OVERHEAD);
    for (int64_t n = 2; n <= 64 && 2 * n <= most; ++n) {
        const int64_t chunks = (most + n - 1) / n;
        const double ctas = (double(T) / (C * chunks) + (R > 1 ? 0.5 * R : 0.0)) * H;
        const double cost = (waves(ctas) + SUM * std::max(1.0, waves(ctas - double(pairs)))) * (chunks + OVERHEAD) +
                            LAUNCHES;
        if (cost < best) {
            best = cost;
            s.tokens = static_cast<int>(chunks * C);
        }
    }
    if (s.tokens) s.slots = static_cast<int>(int64_t(T) / s.tokens + R);
    return s;
}

int launch_chunks(const LinParams &p, int D, int max_query_len, float *ws, const Segments &s, cudaStream_t stream) {
    // Long requests first where CTAs start after others have finished, unless all are about
    // as long: a long one that starts last runs alone at the end.  8 of 65 to 2,048 tokens, 32
    // heads: 113 us with the longest last, 83 first and the others as they come, 78.5 in
    // order; 40 of 65 to 1,000, 8 heads: 72 and 60; 60 of 1 to 300: 48 both.
    const bool sorted = !s.tokens && p.R > 1 && p.R <= kSortedR && int64_t(p.R) * p.H > sm_count() &&
                        4 * int64_t(std::min(max_query_len, p.T)) * p.R > 5 * int64_t(p.T);
    const ChunkParams a{p, ws, s.tokens, s.slots, sorted};
    return D == 128 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace lin
}  // namespace pa
