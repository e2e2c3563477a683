// Paged decode attention with a sliding window and sinks for sm_103a.
//
// The one query of sequence b sits at the newest position L - 1 and sees the
// first S tokens (sinks) and the last W (the window, itself included):
//   o = sum_{j < S or L - W <= j < L} softmax(scale q . k_j) v_j
// Blocks of the table none of whose tokens is visible are never read, so
// their pages may have been freed and their entries may be anything.
//
// Bound: HBM on the visible K/V (a batch), latency (a few sequences).  What
// is read is at most S + W tokens per sequence however long it is, so a
// (sequence, KV head) item is small and the items of a batch are nearly
// equal.  One thread-block cluster of C CTAs computes one item in one launch
// without a workspace: the visible tiles are split evenly over the cluster's
// warps; each warp streams its tiles through its own ring of shared-memory
// stages (as the persistent decode kernel does) with a running maximum and
// sum; the warps' results meet in shared memory, and each CTA sends its part of
// every 1/C of the item's output to the CTA that finishes it (distributed
// shared memory, one cluster barrier).
//
// Measured (bf16, d 128; GPU times, calls replayed from a graph): 64 sequences of
// 128 to 32,768 tokens, window 4096, 32/8 heads: 149 us, 6.8 TB/s (the rate of a
// copy); one sequence of window 1024: 6.2 us (6.4 through the Python call), a
// chain of latencies (launch, length, table, tile, two exchanges).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "pa_decode_tile.cuh"
#include "pa_prefill.cuh"

namespace {

using namespace pa::dec;

constexpr int kNW = 4;  // warps per CTA
constexpr int kMaxCluster = 16;

struct WindowParams {
    void *out;
    const void *q;
    const uint8_t *k_cache, *v_cache;
    const int32_t *block_table, *context_lens;
    int *err;
    int64_t num_blocks;
    int B, Hq, Hkv, bs, bs_log2, MB, window, sinks;
    float qscale;  // scale * log2(e)
};

// DEEP: the deeper ring with fewer CTAs per SM (tensor-core tile only)
template <typename T, int D, int GQ, bool DEEP = false>
struct TileOf {  // CUDA-core tile
    using type = WarpAttn<T, D, GQ>;
    static constexpr bool MMA = false;
    static constexpr int STAGE = Cfg<T, D, GQ>::STAGE;
    // one stage where two take more than 64 KB per CTA: several CTAs per SM
    // instead (24 sequences, window 501, d 64, groups of 1: 7.2 us on the GPU
    // against 8.7).  Stages of 8 KB keep two (64 sequences, window 4096, d 64,
    // groups of 4: 160 us against 194 with one)
    static constexpr int NST = STAGE <= 8192 ? 2 : 1;
    static constexpr int PBUF = 2 * Cfg<T, D, GQ>::TT * GQ * 4;  // p and score buffers, per warp
    static constexpr int MINB = 1;
};
template <int D, int GQ, bool DEEP>
struct TileOf<__nv_bfloat16, D, GQ, DEEP> {  // tensor-core tile
    using type = MmaAttn<D, GQ>;
    static constexpr bool MMA = true;
    static constexpr int STAGE = 2 * MmaCfg<D, GQ>::TILE;
    // Two stages per warp, and as many CTAs per SM as then fit: other CTAs fill
    // the time in which one starts or merges.  32 sequences, window 4096, d 128:
    // 80.5 us with 2 stages and 3 CTAs per SM, 83.4 with 3 and 2, 104.5 with 6
    // and 1; 64 sequences, window 2048, d 64: 43.2 us with 2 stages, 45.6 with
    // 3, 60.2 with 4 (4 KB stages).  DEEP: for the batches of launch().
    static constexpr int NST = DEEP ? (D == 128 ? 3 : 4) : 2;
    static constexpr int PBUF = 0;
    static constexpr int MINB = (D == 128 ? 3 : 4) - (DEEP ? 1 : 0);
};

template <typename T, int D, int GQ, bool DEEP>
struct Layout {
    using TO = TileOf<T, D, GQ, DEEP>;
    static constexpr int WARP = TO::NST * TO::STAGE;  // ring of a warp, then its result
    static constexpr int OFF_P = kNW * WARP;
    // received from the cluster's CTAs: their acc of this CTA's outputs [C][GQ
    // * D / C] and their (max, sum) [C][GQ]
    static constexpr int OFF_CTA = OFF_P + kNW * TO::PBUF;
    static constexpr int OFF_ML = OFF_CTA + GQ * D * 4;
    static constexpr int OFF_WML = OFF_ML + kMaxCluster * GQ * 8;  // the warps' (max, sum) [kNW][GQ]
    static constexpr int OFF_BAR = OFF_WML + kNW * GQ * 8;
    static constexpr int SMEM = OFF_BAR + kNW * TO::NST * 8 + 1024;
    static_assert(GQ * D * 4 <= WARP, "a warp's result must fit its ring");
    static_assert(WARP % 1024 == 0, "swizzled stages must stay aligned");
};

__device__ __forceinline__ uint32_t cluster_ctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_nctarank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_cta(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_cluster2(uint32_t addr, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(addr), "f"(v.x), "f"(v.y)
                 : "memory");
}

template <typename T>
__device__ __forceinline__ void store2(T *dst, float2 v);
template <>
__device__ __forceinline__ void store2<__nv_bfloat16>(__nv_bfloat16 *dst, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(v.x, v.y);
}
template <>
__device__ __forceinline__ void store2<float>(float *dst, float2 v) {
    *reinterpret_cast<float2 *>(dst) = v;
}

// The visible tiles of one sequence: ns sink tiles from token 0, then nw
// window tiles from token wbase; lo is the window's first token.  With the
// window reaching the sinks there is one range from token 0.
struct Visible {
    int L, lo, S, ns, nw, wbase;
    __device__ __forceinline__ int first_token(int t, int TT) const {
        return t < ns ? t * TT : wbase + (t - ns) * TT;
    }
    // visible tokens [a, b) of the TT (or fewer) tokens from tok on of tile t
    __device__ __forceinline__ void rows(int t, int tok, int n, int *a, int *b) const {
        *a = max(0, (t < ns ? 0 : lo) - tok);
        *b = min(n, (t < ns ? S : L) - tok);
    }
};

// A warp's result (max, sum per head, unnormalised acc [GQ][D]) into acc/ml.
template <int D, int GQ>
__device__ __forceinline__ void put_result(MmaAttn<D, GQ> &st, float *acc, float2 *ml) {
    float lh[2];
    st.reduce(lh);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int h = 2 * st.t + j;
        if (h >= GQ) continue;
#pragma unroll
        for (int m = 0; m < D / 16; ++m) {
            acc[h * D + 16 * m + st.g] = st.acc[m][j];
            acc[h * D + 16 * m + st.g + 8] = st.acc[m][2 + j];
        }
        if (st.g == 0) ml[h] = make_float2(st.m_run[j], lh[j]);
    }
}
template <typename T, int D, int GQ>
__device__ __forceinline__ void put_result(WarpAttn<T, D, GQ> &st, float *acc, float2 *ml) {
    float lh[GQ];
    st.reduce(lh);
    st.store_partial(acc, D, reinterpret_cast<float *>(ml), 2, lh);
}

// weight of a partial with maximum m under the common maximum M (0 for an
// empty one; also when every partial is empty)
__device__ __forceinline__ float weight(float m, float M) {
    return m == -INFINITY ? 0.f : exp2f(m - M);
}

template <typename T, int D, int GQ, bool DEEP>
__global__ void __launch_bounds__(kNW * 32, (TileOf<T, D, GQ, DEEP>::MINB))
    decode_window_kernel(const WindowParams p, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap) {
    using TO = TileOf<T, D, GQ, DEEP>;
    using Lay = Layout<T, D, GQ, DEEP>;
    using St = typename TO::type;
    constexpr int TT = St::C::TT;
    constexpr int NST = TO::NST;
    constexpr int ROW = D * int(sizeof(T));
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * Lay::WARP;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR) + warp * NST;
    float *pbuf = reinterpret_cast<float *>(smem + Lay::OFF_P + warp * TO::PBUF);
    float2 *wml = reinterpret_cast<float2 *>(smem + Lay::OFF_WML);
    const int C = cluster_nctarank(), rank = cluster_ctarank();
    const int item = blockIdx.x / C, b = item / p.Hkv, hk = item % p.Hkv;
    if (lane == 0) {
        for (int s = 0; s < NST; ++s) pa::mbar_init(&bars[s], 1);
        pa::fence_barrier_init();
    }
    __syncwarp();
    if (C > 1) cluster_arrive();  // this CTA runs: the others may write to it (waited for below)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- the visible tiles and this warp's share ------------------------------
    Visible vis;
    vis.L = p.context_lens[b];
    const int cap = p.MB << p.bs_log2;
    if (vis.L < 0 || vis.L > cap) {
        if (threadIdx.x == 0) pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
        vis.L = vis.L < 0 ? 0 : cap;
    }
    vis.lo = max(0, vis.L - p.window);
    vis.S = p.sinks;
    if (vis.lo <= vis.S) vis.lo = vis.S = 0;
    vis.ns = (vis.S + TT - 1) / TT;
    vis.wbase = vis.lo / TT * TT;
    vis.nw = (vis.L - vis.wbase + TT - 1) / TT;
    const int nt = vis.ns + vis.nw, parts = C * kNW, part = rank * kNW + warp;
    const int t0 = static_cast<int>(int64_t(nt) * part / parts);
    const int t1 = static_cast<int>(int64_t(nt) * (part + 1) / parts);

    St st;
    st.init(lane);
    st.reset();
    if (t0 < t1)
        st.load_q(static_cast<const T *>(p.q) + (static_cast<size_t>(b) * p.Hq + hk * GQ) * D,
                  p.qscale);

    // ---- block-table entries: 32 (tile, block) slots at a time, one per lane,
    //      the next batch loaded one batch ahead; -1: nothing to copy ----------
    const int nb = max(1, TT >> p.bs_log2), tpb = 32 / nb;  // blocks per tile, tiles per batch
    const int32_t *bt_row = p.block_table + static_cast<size_t>(b) * p.MB;
    auto fetch = [&](int tb) -> int {
        const int t = tb + lane / nb;
        if (t >= t1) return -1;
        const int tok0 = vis.first_token(t, TT), tok = tok0 + (lane % nb) * p.bs;
        int a, e;
        vis.rows(t, tok0, TT, &a, &e);
        // the slot's block covers rows [tok - tok0, tok - tok0 + bs) of the tile
        if (tok - tok0 >= e || (nb > 1 && tok - tok0 + p.bs <= a)) return -1;
        int v = __ldg(bt_row + (tok >> p.bs_log2));
        if (v < 0 || v >= p.num_blocks) {
            pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
            v = 0;
        }
        return v;
    };
    int ent = fetch(t0), ent_next = fetch(t0 + tpb), tb = t0;
    // copies of tile t into its stage (t ascending, each once; whole warp)
    auto issue = [&](int t) {
        if (t - tb >= tpb) {
            tb += tpb;
            ent = ent_next;
            ent_next = fetch(tb + tpb);
        }
        const int s = (t - t0) % NST, slot0 = (t - tb) * nb;
        uint8_t *stage = ring + s * TO::STAGE;
        const uint32_t sk = pa::smem_u32(stage), sv = sk + TO::STAGE / 2;
        const int rows = min(TT, p.bs);  // rows of one copy
        const unsigned live = __ballot_sync(pa::kFull, ent >= 0) >> slot0;
        const int copies = __popc(live & ((1u << nb) - 1u));
        const int r0 = nb > 1 ? 0 : vis.first_token(t, TT) & (p.bs - 1);
        if (lane == 0) pa::mbar_arrive_expect_tx(&bars[s], 2u * copies * rows * ROW);
        for (int j = 0; j < nb; ++j) {
            const int blk = __shfl_sync(pa::kFull, ent, slot0 + j);
            if (lane != 0 || blk < 0) continue;
            const int64_t row = ((static_cast<int64_t>(blk) * p.Hkv + hk) << p.bs_log2) + r0;
            if constexpr (TO::MMA) {
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                    const uint32_t off = h * TT * 128 + j * rows * 128;
                    pa::tma_2d_g2s(sk + off, &kmap, 64 * h, static_cast<int>(row), &bars[s]);
                    pa::tma_2d_g2s(sv + off, &vmap, 64 * h, static_cast<int>(row), &bars[s]);
                }
            } else {
                const uint32_t bytes = static_cast<uint32_t>(rows) * ROW;
                pa::bulk_g2s(stage + j * bytes, p.k_cache + row * ROW, bytes, &bars[s]);
                pa::bulk_g2s(stage + TO::STAGE / 2 + j * bytes, p.v_cache + row * ROW, bytes,
                             &bars[s]);
            }
        }
    };
    for (int t = t0; t < min(t1, t0 + NST); ++t) issue(t);

    bool ok = true;
    for (int t = t0; t < t1; ++t) {
        const int i = t - t0, s = i % NST;
        ok = __all_sync(pa::kFull, pa::mbar_wait(&bars[s], (i / NST) & 1));
        if (!ok) {
            // a copy never completed: record it, wait (bounded) for the others
            // in flight, and meet the other warps with what there is
            if (lane == 0) {
                pa::record_error(p.err, PA_DEVERR_TIMEOUT);
                for (int k = i + 1; k < min(i + NST, t1 - t0); ++k)
                    (void)pa::mbar_wait(&bars[k % NST], (k / NST) & 1);
            }
            __syncwarp();
            break;
        }
        const uint32_t kaddr = pa::smem_u32(ring + s * TO::STAGE);
        int a, e;
        vis.rows(t, vis.first_token(t, TT), TT, &a, &e);
        if constexpr (TO::MMA)
            st.template tile<true>(kaddr, kaddr + TO::STAGE / 2, e, nullptr, nullptr, 0, a);
        else
            st.template tile<true>(kaddr, kaddr + TO::STAGE / 2, e, pbuf, pbuf + TT * GQ, a);
        __syncwarp();
        if (t + NST < t1) {
            pa::fence_proxy_async();
            issue(t + NST);
        }
    }

    // ---- the CTA's result -------------------------------------------------------
    __syncwarp();
    put_result(st, reinterpret_cast<float *>(ring), wml + warp * GQ);
    __syncthreads();
    float *in_acc = reinterpret_cast<float *>(smem + Lay::OFF_CTA);
    float2 *in_ml = reinterpret_cast<float2 *>(smem + Lay::OFF_ML);
    T *out = static_cast<T *>(p.out) + (static_cast<size_t>(b) * p.Hq + hk * GQ) * D;
    const int share = GQ * D / C;  // outputs of a CTA; a multiple of 2: GQ * D >= 64, C <= 16
    if (C > 1) cluster_wait();     // every CTA of the cluster has started
    for (int x = threadIdx.x * 2; x < GQ * D; x += kNW * 64) {
        const int h = x / D;
        float M = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) M = fmaxf(M, wml[w * GQ + h].x);
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
            const float2 ml = wml[w * GQ + h];
            const float f = weight(ml.x, M);
            const float2 v = *reinterpret_cast<const float2 *>(smem + w * Lay::WARP + x * 4);
            l += f * ml.y;
            a = pa::ffma2(make_float2(f, f), v, a);
        }
        if (C == 1) {
            const float inv = vis.L > 0 ? 1.f / l : 0.f;
            store2(out + x, make_float2(a.x * inv, a.y * inv));
        } else {
            const int to = x / share;
            st_cluster2(map_cta(pa::smem_u32(in_acc + rank * share + x % share), to), a);
            if (x % share == 0 || x % D == 0)
                st_cluster2(map_cta(pa::smem_u32(in_ml + rank * GQ + h), to), make_float2(M, l));
        }
    }
    if (C == 1) return;
    // ---- this CTA's outputs ---------------------------------------------------------
    cluster_arrive();
    cluster_wait();  // nothing is sent after this: a CTA may exit before the others
    for (int x = threadIdx.x * 2; x < share; x += kNW * 64) {
        const int h = (rank * share + x) / D;
        float M = -INFINITY, l = 0.f;
        for (int c = 0; c < C; ++c) M = fmaxf(M, in_ml[c * GQ + h].x);
        float2 a = make_float2(0.f, 0.f);
        for (int c = 0; c < C; ++c) {
            const float2 ml = in_ml[c * GQ + h];
            const float2 v = *reinterpret_cast<const float2 *>(in_acc + c * share + x);
            const float f = weight(ml.x, M);
            l += f * ml.y;
            a = pa::ffma2(make_float2(f, f), v, a);
        }
        const float inv = vis.L > 0 ? 1.f / l : 0.f;
        store2(out + rank * share + x, make_float2(a.x * inv, a.y * inv));
    }
}

int sm_count() {
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 0;
    return sms;
}

// CTAs of a kernel that run at once on the current device (0: unknown); looked
// up once per kernel and device.
template <typename K>
int concurrent_ctas(K kern, size_t smem, std::atomic<int> (&cache)[64]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (dev < 64)
        if (const int n = cache[dev].load(std::memory_order_relaxed)) return n;
    int per_sm = 0;
    const int sms = sm_count();
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kNW * 32, smem) != cudaSuccess)
        return 0;
    if (dev < 64) cache[dev].store(per_sm * sms, std::memory_order_relaxed);
    return per_sm * sms;
}

// CTAs of decode_window_kernel that run at once, with its attributes set;
// 0: a CUDA call failed.
template <typename T, int D, int GQ, bool DEEP>
int prepare_kernel() {
    using Lay = Layout<T, D, GQ, DEEP>;
    static std::atomic<uint64_t> smem_done{0};
    static std::atomic<int> slots[64];
    auto kern = decode_window_kernel<T, D, GQ, DEEP>;
    if (pa::pf::set_smem_once(kern, Lay::SMEM, &smem_done)) return 0;
    return concurrent_ctas(kern, Lay::SMEM, slots);
}

template <typename T, int D, int GQ, bool DEEP>
int launch_t(const WindowParams &p, int c, cudaStream_t stream) {
    using TO = TileOf<T, D, GQ, DEEP>;
    using Lay = Layout<T, D, GQ, DEEP>;
    CUtensorMap kmap{}, vmap{};
    if constexpr (TO::MMA) {
        const int64_t rows = (p.num_blocks * p.Hkv) << p.bs_log2;
        const int box = std::min(TO::type::C::TT, p.bs);
        if (int rc = pa::encode_pool_map(&kmap, p.k_cache, rows, D, box)) return rc;
        if (int rc = pa::encode_pool_map(&vmap, p.v_cache, rows, D, box)) return rc;
    }
    const int64_t items = int64_t(p.B) * p.Hkv;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items * c));
    cfg.blockDim = dim3(kNW * 32);
    cfg.dynamicSmemBytes = Lay::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(c), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    (void)cudaGetLastError();  // drop a stale error that is not ours
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, decode_window_kernel<T, D, GQ, DEEP>, p, kmap, vmap);
    if (e != cudaSuccess) return pa::cuda_fail(e, "decode_window launch");
    return pa::check_launch("decode_window launch");
}

template <typename T, int D, int GQ>
int launch(const WindowParams &p, cudaStream_t stream) {
    using TO = TileOf<T, D, GQ>;
    constexpr int TT = TO::type::C::TT;
    const int slots = prepare_kernel<T, D, GQ, false>(), sms = sm_count();
    if (slots <= 0 || sms <= 0)
        return pa::cuda_fail(cudaGetLastError(), "decode_window: kernel attributes");
    // Cluster size: the largest that leaves every warp two tiles (also of the
    // types with one stage, whose warps then wait for each) and all clusters
    // running at once.  A second wave of clusters costs more than the
    // split gains: window 4096, 8 KV heads, 4 sequences: 16.0 us with clusters of
    // 8, 30.4 with 16; 16 sequences of window 1024: 15.9 us with clusters of 2,
    // 21.4 with 4.  One sequence: window 8192 12.1 us with clusters of 16, 18.5
    // with 8.
    static std::atomic<int> cache[64][5];
    const int64_t items = int64_t(p.B) * p.Hkv;
    const int64_t tokens = std::min<int64_t>(int64_t(p.MB) << p.bs_log2, int64_t(p.sinks) + p.window);
    const int64_t tiles = (tokens + TT - 1) / TT;
    int c = 1;
    while (c < kMaxCluster && tiles >= 2 * kNW * 2 * c && items * 2 * c <= slots) {
        const int n = pa::pf::clusters_at_once(decode_window_kernel<T, D, GQ, false>, kNW * 32,
                                               Layout<T, D, GQ, false>::SMEM, 2 * c, cache);
        if (n < 0) return pa::cuda_fail(cudaGetLastError(), "decode_window: occupancy");
        if (items > n) break;
        c *= 2;
    }
    if constexpr (TO::MMA) {
        // A last wave of fewer CTAs than SMs leaves memory idle, each CTA alone
        // on its SM: the time lost, as a part of the whole.  The deeper ring has
        // fewer CTAs at once, so that another number of items ends badly: 512
        // items of window 4096 175 us with two stages (a last wave of 56 CTAs),
        // 150 with the deeper ring (208); 384 items of window 2048 64.6 and 75.2.
        auto lost = [&](int64_t at_once) {
            const int64_t last = items % at_once;
            return items <= at_once || last == 0 || last >= sms ? 0.0 : double(sms - last) / items;
        };
        const int deep = prepare_kernel<T, D, GQ, true>();
        if (deep <= 0) return pa::cuda_fail(cudaGetLastError(), "decode_window: kernel attributes");
        if (c == 1 && lost(slots) > lost(deep) + 0.05)
            return launch_t<T, D, GQ, true>(p, c, stream);
    }
    return launch_t<T, D, GQ, false>(p, c, stream);
}

template <typename T, int D>
int dispatch(int gq, const WindowParams &p, cudaStream_t s) {
    switch (gq) {
        case 1: return launch<T, D, 1>(p, s);
        case 2: return launch<T, D, 2>(p, s);
        case 4: return launch<T, D, 4>(p, s);
        default: return launch<T, D, 8>(p, s);
    }
}

}  // namespace

namespace pa {

// Validate mode of the windowed calls: lengths in [0, capacity] and every
// block with a token visible to the first query (or a later one) in the pool;
// of a prefill also its rows inside [0, total_tokens), no request longer than
// max_query_len.
int validate_window(const int32_t *block_table, int MB, const int32_t *context_lens,
                    const int32_t *query_start, int total_tokens, int max_query_len, int B, int bs,
                    int64_t num_blocks, int window, int sinks, cudaStream_t stream) try {
    std::vector<int32_t> lens(B), table(size_t(B) * MB), qs;
    if (int rc = fetch(lens.data(), context_lens, lens.size() * 4, stream)) return rc;
    if (int rc = fetch(table.data(), block_table, table.size() * 4, stream)) return rc;
    if (query_start) {
        qs.resize(size_t(B) + 1);
        if (int rc = fetch(qs.data(), query_start, qs.size() * 4, stream)) return rc;
    }
    for (int b = 0; b < B; ++b) {
        const int64_t L = lens[b], n = query_start ? int64_t(qs[b + 1]) - qs[b] : 1;
        if (L < 0 || L > int64_t(MB) * bs)
            return fail(PA_ERR_INVALID, "validate: context_lens[%d]=%lld outside [0,%lld]", b,
                        (long long)L, (long long)MB * bs);
        if (query_start && (n < 0 || n > L || n > max_query_len))
            return fail(PA_ERR_INVALID, "validate: request %d has %lld new tokens of %lld, "
                                        "max_query_len %d", b, (long long)n, (long long)L,
                        max_query_len);
        if (query_start && n > 0 && (qs[b] < 0 || qs[b + 1] > total_tokens))
            return fail(PA_ERR_INVALID, "validate: rows [%d,%d) of request %d outside [0,%d)", qs[b],
                        qs[b + 1], b, total_tokens);
        if (L == 0 || n == 0) continue;
        const int64_t lo = std::max<int64_t>(0, L - n - window + 1);
        for (int64_t i = 0; i < (L + bs - 1) / bs; ++i) {
            if (i * bs >= sinks && std::min<int64_t>((i + 1) * bs, L) <= lo) continue;
            const int32_t v = table[size_t(b) * MB + i];
            if (v < 0 || v >= num_blocks)
                return fail(PA_ERR_INVALID, "validate: block_table[%d][%lld]=%d outside pool", b,
                            (long long)i, v);
        }
    }
    return PA_OK;
} catch (const std::bad_alloc &) {
    return fail(PA_ERR_OOM, "validate: host allocation failed");
}

}  // namespace pa

extern "C" int pa_decode_window(void *out, const void *q, const void *k_cache, const void *v_cache,
                                const int32_t *block_table, int max_blocks_per_seq,
                                const int32_t *context_lens, int B, int Hq, int Hkv, int head_dim,
                                int block_size, int64_t num_blocks, float scale, int window,
                                int num_sinks, int dtype, pa_stream_t stream) {
    pa::clear_error();
    if (dtype != PA_BF16 && dtype != PA_F32)
        return pa::fail(PA_ERR_INVALID, "decode_window: bad dtype");
    if (B < 0 || B > 65535 || Hq <= 0 || Hkv <= 0 || Hkv > 1024 || Hq % Hkv || num_blocks <= 0 ||
        max_blocks_per_seq <= 0)
        return pa::fail(PA_ERR_INVALID, "decode_window: bad sizes");
    if (head_dim != 64 && head_dim != 128)
        return pa::fail(PA_ERR_UNSUPPORTED, "decode_window: head_dim %d unsupported", head_dim);
    const int gq = Hq / Hkv;
    if (gq != 1 && gq != 2 && gq != 4 && gq != 8)
        return pa::fail(PA_ERR_UNSUPPORTED, "decode_window: Hq/Hkv=%d unsupported", gq);
    if (!pa::pow2_in(block_size, 8, 128))
        return pa::fail(PA_ERR_UNSUPPORTED, "decode_window: block_size %d unsupported", block_size);
    if (int64_t(max_blocks_per_seq) * block_size > (int64_t(1) << 30))
        return pa::fail(PA_ERR_INVALID, "decode_window: table capacity too large");
    if (num_blocks > INT32_MAX || num_blocks * Hkv * block_size > int64_t(INT32_MAX))
        return pa::fail(PA_ERR_UNSUPPORTED, "decode_window: pools of 2^31 rows or more");
    if (window < 1 || num_sinks < 0)
        return pa::fail(PA_ERR_INVALID, "decode_window: window %d must be positive, num_sinks %d "
                                        "not negative", window, num_sinks);
    if (!(scale > 0.f) || !std::isfinite(scale))
        return pa::fail(PA_ERR_INVALID, "decode_window: scale must be positive and finite");
    if (B == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_table || !context_lens)
        return pa::fail(PA_ERR_INVALID, "decode_window: NULL pointer");
    if (!pa::aligned16(q) || !pa::aligned16(out) || !pa::aligned16(k_cache) ||
        !pa::aligned16(v_cache))
        return pa::fail(PA_ERR_INVALID, "decode_window: q, out and pools must be 16-byte aligned");
    if (pa::validate_on())
        if (int rc = pa::validate_window(block_table, max_blocks_per_seq, context_lens, nullptr, 0,
                                         0, B, block_size, num_blocks, window, num_sinks, stream))
            return rc;
    WindowParams p{};
    p.out = out;
    p.q = q;
    p.k_cache = static_cast<const uint8_t *>(k_cache);
    p.v_cache = static_cast<const uint8_t *>(v_cache);
    p.block_table = block_table;
    p.context_lens = context_lens;
    p.err = pa::device_error_word();
    p.num_blocks = num_blocks;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.bs = block_size;
    while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
    p.MB = max_blocks_per_seq;
    p.window = window;
    p.sinks = num_sinks;
    p.qscale = scale * kLog2e;
    if (dtype == PA_BF16)
        return head_dim == 128 ? dispatch<__nv_bfloat16, 128>(gq, p, stream)
                               : dispatch<__nv_bfloat16, 64>(gq, p, stream);
    return head_dim == 128 ? dispatch<float, 128>(gq, p, stream)
                           : dispatch<float, 64>(gq, p, stream);
}
