// Attention of each request's query rows to an encoder's states in pages (bf16):
// every row of request r sees all L_r states,
//   o = sum_{j < L_r} softmax(scale q . k_j) v_j,   0 where L_r = 0.
//
// Few rows (tokens x query heads of a KV head at most 32: single tokens, beams,
// short chunks): bound by HBM on the states, read once for all rows of their
// (request, KV head).  One thread-block cluster per (request, KV head), its warps
// streaming equal shares of the 16-state tiles through rings of their own, as the
// windowed decode does; the rows are the columns of the warp-level MMA tile, 8 a
// set, up to four sets that use a tile one after another.
// More rows: bound by the tensor cores; the kernels of pa_prefill_window.cuh.
// Where there are more CTAs than run at once, requests with the most states come first:
// one of them that started last would run alone at the end.
//
// Measured: 64 requests of 1 to 5 rows over 400 to 1,500 states (16 KV heads, d 64)
// 41.3 us, 6.1 TB/s (0.89 of HBM; 46.9 in the requests' own order); one row over 1,500
// states 5.1 us on the GPU.  8 requests of 20 to 100 rows over 1,000 to 4,100 states (32/8
// heads, d 128) 41 us: 120 items of up to 65 tiles, two CTAs each (47 with one, of which
// the longest takes it all).  4 of 2,048 rows over 2,000 to 8,192 states 627 to 671 us,
// 1,050 to 1,120 TFLOP/s (0.60 to 0.65 of sustained bf16; tensor pipe 73 % of active cycles).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "pa_cluster.cuh"
#include "pa_decode_tile.cuh"
#include "pa_prefill_window.cuh"

namespace {

using namespace pa::dec;

constexpr int kNW = 4;  // warps per CTA
constexpr int kMaxCluster = 16;
constexpr int kSortedR = 256;  // requests that a CTA puts in order
constexpr int kMaxCols = 32;  // rows of a (request, KV head) that the streaming kernel takes

struct CrossParams {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const int32_t *block_table, *query_start, *encoder_lens;
    int *err;
    int64_t num_blocks;
    int R, T, Hq, Hkv, gq_log2, bs, bs_log2, MB;
    bool sorted;   // more CTAs than run at once: long requests first
    float qscale;  // scale * log2(e)
};

// NG: sets of 8 columns.
template <int D, int NG>
struct CLayout {
    using St = MmaAttn<D, 8>;
    static constexpr int TT = St::C::TT;
    static constexpr int STAGE = 2 * St::C::TILE;
    static constexpr int NST = 2;
    static constexpr int COLS = 8 * NG;
    static constexpr int WARP = NST * STAGE;  // ring of a warp, then its result
    // received from the cluster's CTAs: their acc of this CTA's outputs and their
    // (max, sum) of each column
    static constexpr int OFF_CTA = kNW * WARP;
    static constexpr int OFF_ML = OFF_CTA + COLS * D * 4;
    static constexpr int OFF_WML = OFF_ML + kMaxCluster * COLS * 8;  // the warps' (max, sum)
    static constexpr int OFF_BAR = OFF_WML + kNW * COLS * 8;
    static constexpr int SMEM = OFF_BAR + kNW * NST * 8 + 1024;
    static constexpr int MINB = NG == 4 ? 2 : D == 128 ? 3 : 4;
    static_assert(COLS * D * 4 <= WARP, "a warp's result must fit its ring");
    static_assert(WARP % 1024 == 0, "swizzled stages must stay aligned");
};

template <int D, int NG>
__global__ void __launch_bounds__(kNW * 32, (CLayout<D, NG>::MINB))
    cross_rows_kernel(const CrossParams p, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap) {
    using Lay = CLayout<D, NG>;
    using St = typename Lay::St;
    constexpr int TT = Lay::TT, NST = Lay::NST, ROW = D * 2;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * Lay::WARP;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Lay::OFF_BAR) + warp * NST;
    float2 *wml = reinterpret_cast<float2 *>(smem + Lay::OFF_WML);
    const int C = cluster_nctarank(), rank = cluster_ctarank();
    const int item = blockIdx.x / C, hk = item % p.Hkv;
    int r = item / p.Hkv;
    if (lane == 0) {
        for (int s = 0; s < NST; ++s) pa::mbar_init(&bars[s], 1);
        pa::fence_barrier_init();
    }
    __syncwarp();
    if (C > 1) cluster_arrive();  // this CTA runs: the others may write to it (waited for below)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (p.sorted) {
        // requests with the most states first: the r-th in that order
        __shared__ int lens[kSortedR], found;
        for (int i = threadIdx.x; i < p.R; i += kNW * 32) lens[i] = p.encoder_lens[i];
        __syncthreads();
        for (int i = threadIdx.x; i < p.R; i += kNW * 32) {
            int rank = 0;
            for (int x = 0; x < p.R; ++x) rank += lens[x] > lens[i] || (lens[x] == lens[i] && x < i);
            if (rank == r) found = i;
        }
        __syncthreads();
        r = found;
    }

    const int qs = p.query_start[r], n = p.query_start[r + 1] - qs, cap = p.MB << p.bs_log2;
    int L = p.encoder_lens[r];
    const bool fits = n >= 0 && (n == 0 || (qs >= 0 && n <= p.T - qs)) && n <= Lay::COLS >> p.gq_log2 &&
                      L >= 0 && L <= cap;
    if (!fits && rank == 0 && threadIdx.x == 0) pa::record_error(p.err, PA_DEVERR_BAD_REQUEST);
    const int cols = fits ? n << p.gq_log2 : 0;
    if (cols == 0) {  // the whole cluster
        if (C > 1) cluster_wait();
        return;
    }
    // column c: query token c >> gq_log2, head c & (group - 1) of the KV head's group
    auto row_of = [&](int c) {
        return (static_cast<int64_t>(qs + (c >> p.gq_log2)) * p.Hq + (hk << p.gq_log2) +
                (c & ((1 << p.gq_log2) - 1))) * D;
    };
    // this warp's share of the tiles
    const int nt = (L + TT - 1) / TT, parts = C * kNW, part = rank * kNW + warp;
    const int t0 = static_cast<int>(int64_t(nt) * part / parts);
    const int t1 = static_cast<int>(int64_t(nt) * (part + 1) / parts);

    St st[NG];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        st[j].init(lane);
        st[j].reset();
        const int c = 8 * j + (lane >> 2);
        st[j].load_q_row(t0 < t1 && c < cols ? p.q + row_of(c) : nullptr, p.qscale);
    }

    // ---- block-table entries: 32 (tile, block) slots at a time, one per lane, the
    //      next batch loaded one batch ahead; -1: nothing to copy ------------------
    const int nb = max(1, TT >> p.bs_log2), tpb = 32 / nb;  // blocks per tile, tiles per batch
    const int32_t *bt_row = p.block_table + static_cast<size_t>(r) * p.MB;
    auto fetch = [&](int tb) -> int {
        const int t = tb + lane / nb, tok = t * TT + (lane % nb) * p.bs;
        if (t >= t1 || tok >= L) return -1;
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
        const uint32_t sk = pa::smem_u32(ring + s * Lay::STAGE), sv = sk + Lay::STAGE / 2;
        const int rows = min(TT, p.bs);  // rows of one copy
        const unsigned live = __ballot_sync(pa::kFull, ent >= 0) >> slot0;
        const int copies = __popc(live & ((1u << nb) - 1u));
        const int r0 = nb > 1 ? 0 : (t * TT) & (p.bs - 1);
        if (lane == 0) pa::mbar_arrive_expect_tx(&bars[s], 2u * copies * rows * ROW);
        for (int j = 0; j < nb; ++j) {
            const int blk = __shfl_sync(pa::kFull, ent, slot0 + j);
            if (lane != 0 || blk < 0) continue;
            const int row = ((blk * p.Hkv + hk) << p.bs_log2) + r0;  // (pools below 2^31 rows)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint32_t off = h * TT * 128 + j * rows * 128;
                pa::tma_2d_g2s(sk + off, &kmap, 64 * h, row, &bars[s]);
                pa::tma_2d_g2s(sv + off, &vmap, 64 * h, row, &bars[s]);
            }
        }
    };
    for (int t = t0; t < min(t1, t0 + NST); ++t) issue(t);

    for (int t = t0; t < t1; ++t) {
        const int i = t - t0, s = i % NST;
        if (!__all_sync(pa::kFull, pa::mbar_wait(&bars[s], (i / NST) & 1))) {
            // a copy never completed: record it, wait (bounded) for the others in
            // flight, and meet the other warps with what there is
            if (lane == 0) {
                pa::record_error(p.err, PA_DEVERR_TIMEOUT);
                for (int k = i + 1; k < min(i + NST, t1 - t0); ++k)
                    (void)pa::mbar_wait(&bars[k % NST], (k / NST) & 1);
            }
            __syncwarp();
            break;
        }
        const uint32_t kaddr = pa::smem_u32(ring + s * Lay::STAGE);
#pragma unroll
        for (int j = 0; j < NG; ++j)
            if (j == 0 || 8 * j < cols)
                st[j].template tile<true>(kaddr, kaddr + Lay::STAGE / 2, min(TT, L - t * TT), nullptr, nullptr);
        __syncwarp();
        if (t + NST < t1) {
            pa::fence_proxy_async();
            issue(t + NST);
        }
    }

    // ---- the CTA's result -------------------------------------------------------
    __syncwarp();
    float *racc = reinterpret_cast<float *>(ring);
#pragma unroll
    for (int j = 0; j < NG; ++j) {
        float lh[2];
        st[j].reduce(lh);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 8 * j + 2 * st[j].t + e;
#pragma unroll
            for (int m = 0; m < D / 16; ++m) {
                racc[c * D + 16 * m + st[j].g] = st[j].acc[m][e];
                racc[c * D + 16 * m + st[j].g + 8] = st[j].acc[m][2 + e];
            }
            if (st[j].g == 0) wml[warp * Lay::COLS + c] = make_float2(st[j].m_run[e], lh[e]);
        }
    }
    __syncthreads();
    float *in_acc = reinterpret_cast<float *>(smem + Lay::OFF_CTA);
    float2 *in_ml = reinterpret_cast<float2 *>(smem + Lay::OFF_ML);
    const int share = cols * D / C;  // outputs of a CTA; a multiple of 4: D >= 64, C <= 16
    if (C > 1) cluster_wait();       // every CTA of the cluster has started
    for (int x = threadIdx.x * 2; x < cols * D; x += kNW * 64) {
        const int c = x / D;
        float M = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kNW; ++w) M = fmaxf(M, wml[w * Lay::COLS + c].x);
        float2 a = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kNW; ++w) {
            const float2 ml = wml[w * Lay::COLS + c];
            const float f = weight(ml.x, M);
            const float2 v = *reinterpret_cast<const float2 *>(smem + w * Lay::WARP + x * 4);
            l += f * ml.y;
            a = pa::ffma2(make_float2(f, f), v, a);
        }
        if (C == 1) {
            const float inv = L > 0 ? 1.f / l : 0.f;
            store2(p.out + row_of(c) + x % D, make_float2(a.x * inv, a.y * inv));
        } else {
            const int to = x / share;
            st_cluster2(map_cta(pa::smem_u32(in_acc + rank * share + x % share), to), a);
            if (x % share == 0 || x % D == 0)
                st_cluster2(map_cta(pa::smem_u32(in_ml + rank * Lay::COLS + c), to), make_float2(M, l));
        }
    }
    if (C == 1) return;
    // ---- this CTA's outputs ---------------------------------------------------------
    cluster_arrive();
    cluster_wait();  // nothing is sent after this: a CTA may exit before the others
    for (int x = threadIdx.x * 2; x < share; x += kNW * 64) {
        const int at = rank * share + x, c = at / D;
        float M = -INFINITY, l = 0.f;
        for (int k = 0; k < C; ++k) M = fmaxf(M, in_ml[k * Lay::COLS + c].x);
        float2 a = make_float2(0.f, 0.f);
        for (int k = 0; k < C; ++k) {
            const float2 ml = in_ml[k * Lay::COLS + c];
            const float2 v = *reinterpret_cast<const float2 *>(in_acc + k * share + x);
            const float f = weight(ml.x, M);
            l += f * ml.y;
            a = pa::ffma2(make_float2(f, f), v, a);
        }
        const float inv = L > 0 ? 1.f / l : 0.f;
        store2(p.out + row_of(c) + at % D, make_float2(a.x * inv, a.y * inv));
    }
}

template <int D, int NG>
int launch_rows(const CrossParams &p0, const void *k_cache, const void *v_cache, cudaStream_t stream) {
    using Lay = CLayout<D, NG>;
    auto kern = cross_rows_kernel<D, NG>;
    static std::atomic<uint64_t> done{0};
    if (int rc = pa::pf::set_smem_once(kern, Lay::SMEM, &done)) return rc;
    CUtensorMap kmap, vmap;
    const int64_t rows = (p0.num_blocks * p0.Hkv) << p0.bs_log2;
    const int box = std::min(Lay::TT, p0.bs);
    if (int rc = pa::encode_pool_map(&kmap, k_cache, rows, D, box)) return rc;
    if (int rc = pa::encode_pool_map(&vmap, v_cache, rows, D, box)) return rc;
    // Cluster size: the largest that leaves every warp two tiles and all clusters
    // running at once (as in the windowed decode: a second wave costs more than the
    // split gains).
    static std::atomic<int> cache[64][5];
    const int64_t items = int64_t(p0.R) * p0.Hkv, tiles = (int64_t(p0.MB) << p0.bs_log2) / Lay::TT;
    int c = 1;
    while (c < kMaxCluster && tiles >= 2 * kNW * 2 * c) {
        const int n = pa::pf::clusters_at_once(kern, kNW * 32, Lay::SMEM, 2 * c, cache);
        if (n < 0) return pa::cuda_fail(cudaGetLastError(), "cross_attention: occupancy");
        if (items > n) break;
        c *= 2;
    }
    CrossParams p = p0;
    const int at_once = pa::pf::clusters_at_once(kern, kNW * 32, Lay::SMEM, 1, cache);
    if (at_once < 0) return pa::cuda_fail(cudaGetLastError(), "cross_attention: occupancy");
    p.sorted = items > at_once && p.R > 1 && p.R <= kSortedR;
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p, kmap, vmap);
    if (e != cudaSuccess) return pa::cuda_fail(e, "cross_attention launch");
    return pa::check_launch("cross_attention launch");
}

// Validate mode: rows inside the call, no request longer than max_query_len,
// encoder lengths inside the table and their pages in the pool.
int validate_cross(const CrossParams &p, int max_query_len, cudaStream_t stream) try {
    std::vector<int32_t> lens(p.R), table(size_t(p.R) * p.MB), qs(size_t(p.R) + 1);
    if (int rc = pa::fetch(lens.data(), p.encoder_lens, lens.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(table.data(), p.block_table, table.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(qs.data(), p.query_start, qs.size() * 4, stream)) return rc;
    for (int r = 0; r < p.R; ++r) {
        const int64_t n = int64_t(qs[r + 1]) - qs[r];
        if (n < 0 || n > max_query_len || (n > 0 && (qs[r] < 0 || qs[r + 1] > p.T)))
            return pa::fail(PA_ERR_INVALID, "validate: request %d has rows [%d,%d) of %d, max_query_len %d", r, qs[r],
                            qs[r + 1], p.T, max_query_len);
        if (lens[r] < 0 || lens[r] > int64_t(p.MB) * p.bs)
            return pa::fail(PA_ERR_INVALID, "validate: encoder_lens[%d]=%d outside [0,%lld]", r, lens[r],
                            (long long)p.MB * p.bs);
        for (int64_t i = 0; n > 0 && i < (int64_t(lens[r]) + p.bs - 1) / p.bs; ++i) {
            const int32_t v = table[size_t(r) * p.MB + i];
            if (v < 0 || v >= p.num_blocks)
                return pa::fail(PA_ERR_INVALID, "validate: block_table[%d][%lld]=%d outside pool", r, (long long)i, v);
        }
    }
    return PA_OK;
} catch (const std::bad_alloc &) {
    return pa::fail(PA_ERR_OOM, "validate: host allocation failed");
}

}  // namespace

extern "C" int pa_cross_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *block_table, int max_blocks_per_seq, const int32_t *query_start,
                                  const int32_t *encoder_lens, int R, int total_tokens, int max_query_len, int Hq,
                                  int Hkv, int head_dim, int block_size, int64_t num_blocks, float scale, int dtype,
                                  pa_stream_t stream) {
    pa::clear_error();
    if (dtype != PA_BF16)
        return pa::fail(dtype == PA_F32 ? PA_ERR_UNSUPPORTED : PA_ERR_INVALID, "cross_attention: bf16 only");
    if (R < 0 || R > 65535 || total_tokens < 0 || max_query_len < 0 || Hq <= 0 || Hkv <= 0 || Hkv > 1024 ||
        Hq % Hkv || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return pa::fail(PA_ERR_INVALID, "cross_attention: bad sizes");
    if (head_dim != 64 && head_dim != 128)
        return pa::fail(PA_ERR_UNSUPPORTED, "cross_attention: head_dim %d unsupported", head_dim);
    const int gq = Hq / Hkv;
    if (gq != 1 && gq != 2 && gq != 4 && gq != 8)
        return pa::fail(PA_ERR_UNSUPPORTED, "cross_attention: Hq/Hkv=%d unsupported", gq);
    if (!pa::pow2_in(block_size, 8, 128))
        return pa::fail(PA_ERR_UNSUPPORTED, "cross_attention: block_size %d unsupported", block_size);
    if (int64_t(max_blocks_per_seq) * block_size > (int64_t(1) << 30))
        return pa::fail(PA_ERR_INVALID, "cross_attention: table capacity too large");
    if (num_blocks > INT32_MAX || num_blocks * Hkv * block_size > int64_t(INT32_MAX) - 256)
        return pa::fail(PA_ERR_UNSUPPORTED, "cross_attention: pools of 2^31 rows or more");
    // items are counted in 32 bits: (tokens / 16 + requests) * KV heads
    if ((int64_t(total_tokens) / 16 + std::min(R, pa::win::kMaxR)) * Hkv > INT32_MAX / 2)
        return pa::fail(PA_ERR_UNSUPPORTED, "cross_attention: too many query tokens");
    if (!(scale > 0.f) || !std::isfinite(scale))
        return pa::fail(PA_ERR_INVALID, "cross_attention: scale must be positive and finite");
    if (R == 0 || total_tokens == 0 || max_query_len == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_table || !query_start || !encoder_lens)
        return pa::fail(PA_ERR_INVALID, "cross_attention: NULL pointer");
    if (!pa::aligned16(q) || !pa::aligned16(out) || !pa::aligned16(k_cache) || !pa::aligned16(v_cache))
        return pa::fail(PA_ERR_INVALID, "cross_attention: q, out and pools must be 16-byte aligned");
    CrossParams c{};
    c.out = static_cast<__nv_bfloat16 *>(out);
    c.q = static_cast<const __nv_bfloat16 *>(q);
    c.block_table = block_table;
    c.query_start = query_start;
    c.encoder_lens = encoder_lens;
    c.num_blocks = num_blocks;
    c.R = R;
    c.T = total_tokens;
    c.Hq = Hq;
    c.Hkv = Hkv;
    c.gq_log2 = pa::pf::log2_int(gq);
    c.bs = block_size;
    c.bs_log2 = pa::pf::log2_int(block_size);
    c.MB = max_blocks_per_seq;
    c.qscale = scale * kLog2e;
    if (pa::validate_on())
        if (int rc = validate_cross(c, max_query_len, stream)) return rc;
    c.err = pa::device_error_word();
    const int64_t cols = int64_t(std::min(max_query_len, total_tokens)) * gq;  // (a bound may be generous)
    if (cols <= kMaxCols) {
        auto pick = [&](auto d) -> int {
            constexpr int DD = decltype(d)::value;
            if (cols <= 8) return launch_rows<DD, 1>(c, k_cache, v_cache, stream);
            if (cols <= 16) return launch_rows<DD, 2>(c, k_cache, v_cache, stream);
            return launch_rows<DD, 4>(c, k_cache, v_cache, stream);
        };
        return head_dim == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 64>{});
    }
    pa::win::WinParams p{};
    p.out = c.out;
    p.block_table = block_table;
    p.query_start = query_start;
    p.context_lens = encoder_lens;
    p.err = c.err;
    p.num_blocks = num_blocks;
    p.R = R;
    p.T = total_tokens;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.bs = block_size;
    p.bs_log2 = c.bs_log2;
    p.MB = max_blocks_per_seq;
    p.window = 1 << 30;  // every state, and no sinks
    p.qscale = c.qscale;
    auto pick = [&](auto d) -> int {
        constexpr int DD = decltype(d)::value;
        switch (gq) {
            case 1: return pa::win::launch<DD, 1, true>(p, q, k_cache, v_cache, max_query_len, stream);
            case 2: return pa::win::launch<DD, 2, true>(p, q, k_cache, v_cache, max_query_len, stream);
            case 4: return pa::win::launch<DD, 4, true>(p, q, k_cache, v_cache, max_query_len, stream);
            default: return pa::win::launch<DD, 8, true>(p, q, k_cache, v_cache, max_query_len, stream);
        }
    };
    return head_dim == 128 ? pick(std::integral_constant<int, 128>{}) : pick(std::integral_constant<int, 64>{});
}
