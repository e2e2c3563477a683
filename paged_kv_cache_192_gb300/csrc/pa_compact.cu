// Compaction of paged sequences: each KV head keeps some of a sequence's
// tokens, and their K and V rows move to the front of the sequence, in place
// or into other pages.  Row i of (sequence b, head h) becomes the old row
// keep[b][h][i]; nothing is computed, so the bytes are the old ones.
//
// Bound: memory (each kept row is read and written once: 4 rows per token and
// head with K and V).
//
// In place, a row that is read may lie where an earlier row is written.  The
// positions are ascending, so row i comes from position keep[i] >= i: the rows
// of a (sequence, head, cache) are walked in order in chunks of rows [i0, i1);
// a chunk is read (cp.async) into a ring of stages in shared memory and
// written after a barrier behind its arrival.  Later chunks read positions
// >= i1 only, which this chunk does not write, and what it overwrites was read
// by this chunk or an earlier one; so the reads of the next chunks are in
// flight while a chunk is written, and only a barrier per chunk holds the
// threads together.  Positions and pages are looked up once per row (not per
// piece), 512 rows at a time and one batch ahead.  One CTA walks a list when
// there are many; a cluster of CTAs takes larger chunks together (its barrier
// in the CTA barrier's place) when there are few.
//
// Measured (bf16, d 128, 8 KV heads): 64 sequences keeping about 4,000 tokens,
// 2.1 GB read and written, 330 us, 0.94 of the copy rate; before the ring, with rows
// held in registers and looked up per piece, 0.67 to 0.77.
#include <atomic>
#include <new>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_prefill.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;    // 16-byte pieces of a thread in a stage
constexpr int kStages = 4;
constexpr int kMeta = 512;  // rows whose pages are looked up at a time (two per thread)
constexpr int kSmem = kStages * kRows * kThreads * 16 + 2 * kMeta * 8;
static_assert(kMeta == 2 * kThreads, "two rows per thread");
// a row has at least 8 lanes, so a batch of looked-up rows spans several chunks
static_assert(kMeta / (kRows * kThreads / 8) >= kStages, "a batch ahead of the reads");

struct CompactParams {
    uint8_t *k_cache, *v_cache;
    const int32_t *src_table, *dst_table, *keep, *keep_lens;
    int64_t num_blocks;
    int Hkv, bs, bs_log2, MBs, MBd, max_keep;
    int row, row_log2;  // 16-byte pieces of a row; lanes of a row: a power of two, 8 or more
    int *err;
};

__device__ __forceinline__ void sync_readers(bool cluster) {
    if (cluster) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    } else {
        __syncthreads();
    }
}

// grid: x = (sequence, KV head) x CTA of the cluster, y = cache (0: K, 1: V)
template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p) {
    extern __shared__ __align__(128) uint8_t ring[];  // [kStages][kRows][kThreads] pieces
    // pool rows (from, to) of two batches of rows; to < 0: nothing to move
    int2(*meta)[kMeta] = reinterpret_cast<int2(*)[kMeta]>(ring + kStages * kRows * kThreads * 16);
    uint32_t C = 1, rank = 0;
    if (CLUSTER) {
        asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
        asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int list = blockIdx.x / C, b = list / p.Hkv, h = list % p.Hkv;
    uint4 *pool = reinterpret_cast<uint4 *>(blockIdx.y ? p.v_cache : p.k_cache);
    int n = p.keep_lens[b];
    const int cap = min(p.max_keep, p.MBd << p.bs_log2), src_cap = p.MBs << p.bs_log2;
    if (n < 0 || n > cap) {
        if (threadIdx.x == 0) pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
        n = n < 0 ? 0 : cap;
    }
    const int32_t *keep = p.keep + static_cast<int64_t>(list) * p.max_keep;
    const int32_t *src_row = p.src_table + static_cast<int64_t>(b) * p.MBs;
    const int32_t *dst_row = p.dst_table + static_cast<int64_t>(b) * p.MBd;
    const int rpp_log2 = 8 - p.row_log2;          // rows of one pass of the 256 threads
    const int R = kRows << rpp_log2, chunk = C * R;  // rows of a chunk: the CTA's, the cluster's
    const int batch = kMeta / R;                  // chunks of a batch
    const int nchunks = (n + chunk - 1) / chunk;
    const int col = threadIdx.x & ((1 << p.row_log2) - 1), sub = threadIdx.x >> p.row_log2;
    const bool idle = col >= p.row;

    // row i of the list that the CTA's row m of batch k is; >= n: none
    auto list_row = [&](int k, int m) { return (k * batch + m / R) * chunk + int(rank) * R + m % R; };
    // pool row of token j of this head under a table row; -1: no such page
    auto row_of = [&](const int32_t *table, int j) -> int {
        const int blk = __ldg(table + (j >> p.bs_log2));
        if (blk < 0 || blk >= p.num_blocks) return -1;
        return ((blk * p.Hkv + h) << p.bs_log2) + (j & (p.bs - 1));
    };
    int kept[2];  // of the batch after `rows`
    int2 rows[2];
    auto load_kept = [&](int k) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = list_row(k, threadIdx.x + u * kThreads);
            kept[u] = i >= 0 && i < n ? __ldg(keep + i) : -1;
        }
    };
    auto load_rows = [&](int k) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = list_row(k, threadIdx.x + u * kThreads), j = kept[u];
            rows[u] = make_int2(-1, -1);
            if (i < 0 || i >= n) continue;
            const int from = j >= 0 && j < src_cap ? row_of(src_row, j) : -1;
            const int to = row_of(dst_row, i);
            if (from < 0 || to < 0) pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
            else if (from != to) rows[u] = make_int2(from, to);
        }
    };
    auto put_rows = [&](int k) {
#pragma unroll
        for (int u = 0; u < 2; ++u) meta[k & 1][threadIdx.x + u * kThreads] = rows[u];
    };
    auto row_of_chunk = [&](int q, int k) -> int2 {
        return meta[(q / batch) & 1][(q % batch) * R + (k << rpp_log2) + sub];
    };
    auto piece = [&](int q, int k) {
        return ring + (((q % kStages) * kRows + k) * kThreads + threadIdx.x) * 16;
    };
    auto issue = [&](int q) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int2 r = q < nchunks ? row_of_chunk(q, k) : make_int2(-1, -1);
            if (r.y >= 0 && !idle)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 pa::smem_u32(piece(q, k))),
                             "l"(pool + static_cast<int64_t>(r.x) * p.row + col)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    load_kept(0);
    load_rows(0);
    load_kept(1);
    put_rows(0);
    load_rows(1);
    load_kept(2);
    __syncthreads();
    for (int q = 0; q < kStages - 1; ++q) issue(q);
    for (int q = 0; q < nchunks; ++q) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
        sync_readers(CLUSTER);
        if (q % batch == 0) {
            // every thread is past the batch before this one: its rows make way
            // for those of the next, which the reads reach after another barrier
            const int k = q / batch;
            put_rows(k + 1);
            load_rows(k + 2);
            load_kept(k + 3);
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int2 r = row_of_chunk(q, k);
            if (r.y >= 0 && !idle)
                pool[static_cast<int64_t>(r.y) * p.row + col] =
                    *reinterpret_cast<const uint4 *>(piece(q, k));
        }
        issue(q + kStages - 1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Validate mode: kept positions ascending and inside the source pages, pages
// inside the pool, no page written for two rows of the batch, and a page that
// is written read only in place (same sequence, same logical block).
int validate_compact(const int32_t *src_table, const int32_t *dst_table, const int32_t *keep,
                     const int32_t *keep_lens, int B, int Hkv, int MBs, int MBd, int max_keep,
                     int bs, int64_t num_blocks, cudaStream_t stream) try {
    std::vector<int32_t> n(B), st(size_t(B) * MBs), dt(size_t(B) * MBd),
        kp(size_t(B) * Hkv * max_keep);
    if (int rc = pa::fetch(n.data(), keep_lens, n.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(st.data(), src_table, st.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(dt.data(), dst_table, dt.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(kp.data(), keep, kp.size() * 4, stream)) return rc;
    std::unordered_map<int32_t, int64_t> written;  // page -> row * 2^32 + logical block
    for (int b = 0; b < B; ++b) {
        if (n[b] < 0 || n[b] > max_keep || int64_t(n[b]) > int64_t(MBd) * bs)
            return pa::fail(PA_ERR_INVALID, "validate: keep_lens[%d]=%d", b, n[b]);
        for (int i = 0; i < (n[b] + bs - 1) / bs; ++i) {
            const int32_t v = dt[size_t(b) * MBd + i];
            if (v < 0 || v >= num_blocks)
                return pa::fail(PA_ERR_INVALID, "validate: dst_table[%d][%d]=%d outside pool", b, i, v);
            if (!written.emplace(v, (int64_t(b) << 32) + i).second)
                return pa::fail(PA_ERR_INVALID, "validate: page %d is written twice", v);
        }
    }
    for (int b = 0; b < B; ++b)
        for (int h = 0; h < Hkv; ++h) {
            int64_t last = -1;
            for (int i = 0; i < n[b]; ++i) {
                const int64_t j = kp[(size_t(b) * Hkv + h) * max_keep + i];
                if (j <= last || j >= int64_t(MBs) * bs)
                    return pa::fail(PA_ERR_INVALID,
                                    "validate: keep[%d][%d][%d]=%lld (ascending, inside the table)",
                                    b, h, i, (long long)j);
                last = j;
                const int32_t v = st[size_t(b) * MBs + j / bs];
                if (v < 0 || v >= num_blocks)
                    return pa::fail(PA_ERR_INVALID, "validate: src_table[%d][%lld]=%d outside pool",
                                    b, (long long)(j / bs), v);
                const auto it = written.find(v);
                if (it != written.end() && it->second != (int64_t(b) << 32) + j / bs)
                    return pa::fail(PA_ERR_INVALID,
                                    "validate: page %d is read for row %d and written elsewhere", v, b);
            }
        }
    return PA_OK;
} catch (const std::bad_alloc &) {
    return pa::fail(PA_ERR_OOM, "validate: host allocation failed");
}

}  // namespace

extern "C" int pa_compact_cache(void *k_cache, void *v_cache, const int32_t *src_table,
                                int src_blocks_per_seq, const int32_t *dst_table,
                                int dst_blocks_per_seq, const int32_t *keep, int max_keep,
                                const int32_t *keep_lens, int B, int64_t num_blocks, int Hkv,
                                int block_size, int head_dim, int dtype, pa_stream_t stream) {
    pa::clear_error();
    const int es = static_cast<int>(pa::dtype_size(dtype));
    if (!es) return pa::fail(PA_ERR_INVALID, "compact_cache: bad dtype %d", dtype);
    if (B < 0 || B > 65535 || num_blocks <= 0 || Hkv <= 0 || Hkv > 1024 || head_dim <= 0 ||
        head_dim > 1024 || max_keep < 0 || src_blocks_per_seq <= 0 || dst_blocks_per_seq <= 0)
        return pa::fail(PA_ERR_INVALID, "compact_cache: bad sizes");
    if (!pa::pow2_in(block_size, 1, 1024))
        return pa::fail(PA_ERR_INVALID, "compact_cache: block_size must be a power of two");
    if (int64_t(src_blocks_per_seq) * block_size > (int64_t(1) << 30) ||
        int64_t(dst_blocks_per_seq) * block_size > (int64_t(1) << 30) || max_keep > (1 << 30))
        return pa::fail(PA_ERR_INVALID, "compact_cache: table capacity too large");
    if (num_blocks > INT32_MAX || num_blocks * Hkv * block_size > int64_t(INT32_MAX))
        return pa::fail(PA_ERR_UNSUPPORTED, "compact_cache: pools of 2^31 rows or more");
    if ((head_dim * es) % 16)
        return pa::fail(PA_ERR_INVALID, "compact_cache: row bytes must be a multiple of 16");
    if (B == 0 || max_keep == 0) return PA_OK;
    if (!k_cache || !v_cache || !src_table || !dst_table || !keep || !keep_lens)
        return pa::fail(PA_ERR_INVALID, "compact_cache: NULL pointer");
    if (!pa::aligned16(k_cache) || !pa::aligned16(v_cache))
        return pa::fail(PA_ERR_INVALID, "compact_cache: pools must be 16-byte aligned");
    if (pa::validate_on())
        if (int rc = validate_compact(src_table, dst_table, keep, keep_lens, B, Hkv,
                                      src_blocks_per_seq, dst_blocks_per_seq, max_keep, block_size,
                                      num_blocks, stream))
            return rc;
    CompactParams p{};
    p.k_cache = static_cast<uint8_t *>(k_cache);
    p.v_cache = static_cast<uint8_t *>(v_cache);
    p.src_table = src_table;
    p.dst_table = dst_table;
    p.keep = keep;
    p.keep_lens = keep_lens;
    p.num_blocks = num_blocks;
    p.Hkv = Hkv;
    p.bs = block_size;
    while ((1 << p.bs_log2) < block_size) ++p.bs_log2;
    p.MBs = src_blocks_per_seq;
    p.MBd = dst_blocks_per_seq;
    p.max_keep = max_keep;
    p.row = head_dim * es / 16;
    p.err = pa::device_error_word();
    p.row_log2 = 3;
    while ((1 << p.row_log2) < p.row) ++p.row_log2;
    // Clusters only when the lists alone are fewer than 3/4 of the SMs: a
    // cluster's barrier costs more than a CTA's.  4,000 of 9,000 tokens, 8 KV
    // heads, with clusters of up to 8 against one CTA per list: 2 sequences (32
    // lists) 19.8 / 40.5 us, 4 (64) 36.2 / 43.1, 8 (128) 58.0 / 51.9.
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return pa::cuda_fail(cudaGetLastError(), "compact_cache: SM count");
    const int64_t lists = int64_t(B) * Hkv;
    const int rows = kThreads >> p.row_log2;  // of one pass of a CTA
    unsigned c = 1;
    if (lists * 8 < 3 * sms)
        while (c < 8 && int64_t(rows) * kRows * c < max_keep) c *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(lists) * c, 2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {c, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = c > 1 ? 2 : 1;
    (void)cudaGetLastError();  // drop a stale error that is not ours
    auto kern = c > 1 ? compact_kernel<true> : compact_kernel<false>;
    static std::atomic<uint64_t> smem_done[2];
    if (int rc = pa::pf::set_smem_once(kern, kSmem, &smem_done[c > 1])) return rc;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e != cudaSuccess) return pa::cuda_fail(e, "compact_cache launch");
    return pa::check_launch("compact_cache launch");
}
