// Compaction of paged sequences: each KV head keeps some of a sequence's
// tokens, and their K and V rows move to the front of the sequence, in place
// or into other pages.  Row i of (sequence b, head h) becomes the old row
// keep[b][h][i]; nothing is computed, so the bytes are the old ones.
//
// Bound: memory (each kept row is read and written once: 4 rows per token and
// head with K and V).
//
// In place, a row that is read may lie where an earlier row is written.  The
// positions are ascending, so row i comes from position keep[i] >= i: one CTA
// walks the rows of its (sequence, head, cache, column slice) in order, reads
// a chunk of rows [i0, i1) into registers, and writes it after a barrier.
// Later chunks read positions >= i1 only, which this chunk does not write,
// and what it overwrites was read by this chunk or an earlier one.
#include <new>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 8;  // 16-byte pieces in flight per thread

struct CompactParams {
    uint8_t *k_cache, *v_cache;
    const int32_t *src_table, *dst_table, *keep, *keep_lens;
    int64_t num_blocks;
    int Hkv, bs, bs_log2, MBs, MBd, max_keep, row, slice;  // row, slice: 16-byte pieces
    int *err;
};

// grid: x = (sequence, KV head), y = cache (0: K, 1: V), z = column slice
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
    uint4 *pool = reinterpret_cast<uint4 *>(blockIdx.y ? p.v_cache : p.k_cache);
    int n = p.keep_lens[b];
    const int cap = min(p.max_keep, p.MBd << p.bs_log2);
    if (n < 0 || n > cap) {
        if (threadIdx.x == 0) pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
        n = n < 0 ? 0 : cap;
    }
    const int32_t *keep = p.keep + static_cast<int64_t>(blockIdx.x) * p.max_keep;
    const int32_t *src_row = p.src_table + static_cast<int64_t>(b) * p.MBs;
    const int32_t *dst_row = p.dst_table + static_cast<int64_t>(b) * p.MBd;
    const int col = blockIdx.z * p.slice + threadIdx.x % p.slice;
    const int rpp = kThreads / p.slice;  // rows of one pass of the CTA
    // piece of token j of this head under table row `t`; -1: no such page
    auto piece = [&](const int32_t *t, int j) -> int64_t {
        const int blk = t[j >> p.bs_log2];
        if (blk < 0 || blk >= p.num_blocks) return -1;
        const int64_t r = ((static_cast<int64_t>(blk) * p.Hkv + h) << p.bs_log2) + (j & (p.bs - 1));
        return r * p.row + col;
    };
    for (int i0 = 0; i0 < n; i0 += kRows * rpp) {
        uint4 v[kRows];
        int64_t to[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int i = i0 + k * rpp + threadIdx.x / p.slice;
            to[k] = -1;
            if (i >= n || col >= p.row) continue;
            const int j = keep[i];
            if (j < 0 || j >= p.MBs << p.bs_log2) {
                pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
                continue;
            }
            const int64_t from = piece(src_row, j);
            to[k] = piece(dst_row, i);
            if (from < 0 || to[k] < 0) {
                pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
                to[k] = -1;
            } else if (from == to[k]) {
                to[k] = -1;  // stays where it is
            } else {
                v[k] = pool[from];
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (to[k] >= 0) pool[to[k]] = v[k];
    }
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
    // columns: the whole row when there are enough (sequence, head) pairs to
    // fill the GPU, else slices of at least four pieces (64 bytes)
    p.slice = 1;
    while (p.slice < p.row && p.slice < kThreads) p.slice *= 2;
    auto slices = [&] { return (p.row + p.slice - 1) / p.slice; };
    while (p.slice > 4 && int64_t(B) * Hkv * 2 * slices() < 2 * 152) p.slice /= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(B * Hkv), 2, static_cast<unsigned>(slices()));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    (void)cudaGetLastError();  // drop a stale error that is not ours
    const cudaError_t e = cudaLaunchKernelEx(&cfg, compact_kernel, p);
    if (e != cudaSuccess) return pa::cuda_fail(e, "compact_cache launch");
    return pa::check_launch("compact_cache launch");
}
