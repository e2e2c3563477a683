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
#include "pa_prefill_window.cuh"

namespace {

using namespace pa::win;

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
            case 1: return launch<DD, 1, false>(p, q, k_cache, v_cache, max_query_len, stream);
            case 2: return launch<DD, 2, false>(p, q, k_cache, v_cache, max_query_len, stream);
            case 4: return launch<DD, 4, false>(p, q, k_cache, v_cache, max_query_len, stream);
            default: return launch<DD, 8, false>(p, q, k_cache, v_cache, max_query_len, stream);
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
