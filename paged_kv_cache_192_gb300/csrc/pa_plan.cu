// A serving step's block tables, slots and positions from its requests'
// lengths, with the pages taken from and given back to a pool on the device.
//
// Row r of the step is sequence s with L tokens that becomes L' = max(0, L + c)
// long: b = ceil(L / bs) pages become b' = ceil(L' / bs).  Pages taken come from
// the front of the ring of free pages, row by row (exclusive prefix sums of the
// rows' b' - b), pages given up go behind its end.  The new token t of the step
// belongs to the row whose range of the prefix sum of the c holds it, at position
// p = L + t - start and slot page[p / bs] * bs + p % bs.
//
// Bound: latency.  A table entry is 4 bytes in and 4 out and a token 16 bytes
// out, so even 1,024 tables of 2,048 entries move 12 MB; the rest is one launch
// and a chain of dependent loads (ids, lengths, pages).  One launch: every CTA
// repeats the prefix sums of all rows (a few thousand numbers, from L2) instead
// of waiting for a launch that makes them, then writes its share of the tables
// and tokens.  No CTA writes what another may still read: new pages lie behind
// the old ones, given pages behind the ring's end, and the lengths and the ring's
// ends are advanced by the CTA that finishes last (a ticket in the ring's state).
//
// Measured: a step of 64 sequences with tables of 260 entries 4.2 us on the GPU (6.2
// through the Python call), 1,024 sequences with tables of 2,048 entries and 20 tokens
// each 9.5 us.
#include <algorithm>
#include <atomic>
#include <new>
#include <vector>

#include "pa_prefill.cuh"

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxRows = 4096;         // rows of a step (tables in shared memory)
constexpr int kMaxSeqs = 1 << 19;      // one bit each in shared memory
constexpr unsigned kMany = 0x7fffffff;  // where sums saturate: more than any limit

struct PlanParams {
    const int32_t *seq_ids, *change;
    int32_t *pages, *lens, *ring, *state;
    int32_t *table, *context_lens, *query_start;
    int64_t *slots, *positions;
    int *err;
    int R, S, MB, W, NB, bs_log2, max_tokens;
    bool vec;  // 16-byte accesses of both tables' rows
};

// A row as every CTA sees it; `taken`, `given` and `start` are the sums of the
// rows before it.
struct Row {
    int seq, old_len, new_len;
    unsigned taken, given, start;
};

// Sums that do not fit stay at kMany; as no term is negative the order of the
// additions does not matter.
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, kMany); }

struct Sums {
    unsigned taken, given, start;
    __device__ __forceinline__ void add(const Sums &o) {
        taken = sat_add(taken, o.taken);
        given = sat_add(given, o.given);
        start = sat_add(start, o.start);
    }
};

__global__ void __launch_bounds__(kThreads) plan_step_kernel(const PlanParams p) {
    extern __shared__ uint8_t smem[];
    Row *rows = reinterpret_cast<Row *>(smem);
    unsigned *seen = reinterpret_cast<unsigned *>(rows + p.R);  // a bit per sequence
    __shared__ Sums warp_sums[kWarps];
    __shared__ int bad, last;  // PA_DEVERR_* bits of a step that is refused
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int bs_log2 = p.bs_log2, bs1 = (1 << bs_log2) - 1;
    auto blocks = [&](int len) { return static_cast<int>((static_cast<int64_t>(len) + bs1) >> bs_log2); };
    const int cap = min(p.MB, p.W);  // blocks that a row's sequence may have

    for (int i = tid; i < (p.S + 31) / 32; i += kThreads) seen[i] = 0;
    if (tid == 0) bad = 0;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- the rows and their prefix sums ------------------------------------------
    const int first = p.state[0], count = p.state[1];
    Sums total{0, 0, 0};
    constexpr int PER = kMaxRows / kThreads;  // rows of a thread: two latencies for all of them
    int id[PER], change[PER], len[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int r = k * kThreads + tid;
        id[k] = r < p.R ? p.seq_ids[r] : -1;
        change[k] = r < p.R ? p.change[r] : 0;
    }
#pragma unroll
    for (int k = 0; k < PER; ++k) len[k] = id[k] >= 0 && id[k] < p.S ? p.lens[id[k]] : 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        if (k * kThreads >= p.R) break;
        const int r = k * kThreads + tid;
        Row row{-1, 0, 0, 0, 0, 0};
        Sums x{0, 0, 0};
        if (r < p.R) {
            const int s = id[k], c = change[k], L = len[k];
            if (s >= p.S) {
                atomicOr(&bad, PA_DEVERR_BAD_REQUEST);
            } else if (s >= 0) {
                if (L < 0 || blocks(L) > p.MB) {
                    atomicOr(&bad, PA_DEVERR_BAD_REQUEST);
                } else {
                    const int64_t n = max(static_cast<int64_t>(L) + c, int64_t(0));
                    row.seq = s;
                    row.old_len = row.new_len = L;
                    // (which of two rows of a sequence comes second does not show: the step is
                    // refused and both keep what there is)
                    if (atomicOr(&seen[s >> 5], 1u << (s & 31)) >> (s & 31) & 1) atomicOr(&bad, PA_DEVERR_BAD_REQUEST);
                    if ((n + bs1) >> bs_log2 > cap) {
                        atomicOr(&bad, PA_DEVERR_NO_BLOCKS);
                    } else {
                        const int b0 = blocks(L), b1 = blocks(static_cast<int>(n));
                        row.new_len = static_cast<int>(n);
                        x = Sums{static_cast<unsigned>(max(b1 - b0, 0)), static_cast<unsigned>(max(b0 - b1, 0)),
                                 static_cast<unsigned>(max(row.new_len - L, 0))};
                    }
                }
            }
        }
        Sums incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums y{__shfl_up_sync(pa::kFull, incl.taken, o), __shfl_up_sync(pa::kFull, incl.given, o),
                         __shfl_up_sync(pa::kFull, incl.start, o)};
            if (lane >= o) incl.add(y);
        }
        if (lane == 31) warp_sums[warp] = incl;
        __syncthreads();
        Sums before = total;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before.add(warp_sums[w]);
            total.add(warp_sums[w]);
        }
        // (below kMany unless the step is refused, so the differences are exact)
        if (r < p.R) {
            before.add(incl);
            row.taken = before.taken - x.taken;
            row.given = before.given - x.given;
            row.start = before.start - x.start;
            rows[r] = row;
        }
        __syncthreads();
    }
    // All or nothing: what does not fit changes nothing.  (That many pages given
    // back cannot be free already: the state is not what this call left there.)
    int why = bad;
    if (first < 0 || first >= p.NB || count < 0 || count > p.NB ||
        static_cast<unsigned>(count) + total.given > static_cast<unsigned>(p.NB))
        why |= PA_DEVERR_BAD_REQUEST;
    else if (total.taken > static_cast<unsigned>(count) || total.start > static_cast<unsigned>(p.max_tokens))
        why |= PA_DEVERR_NO_BLOCKS;
    if (why) {
        for (int r = tid; r < p.R; r += kThreads) {
            const int L = rows[r].old_len;
            // a table that is too narrow for what the sequence holds shows nothing of it
            rows[r].new_len = rows[r].old_len = blocks(L) <= cap ? L : 0;
            rows[r].taken = rows[r].given = rows[r].start = 0;
        }
        total = Sums{0, 0, 0};
        __syncthreads();
    }
    auto wrap = [&](int i) { return i >= p.NB ? i - p.NB : i; };  // (sums of two numbers up to NB)

    // ---- tables and tokens: units of a warp, some at once so that their loads overlap ----
    constexpr int AT_ONCE = 2;
    // Unit u: 128 entries of a row, u < p.R * chunks; then 32 tokens.
    const int chunks = (max(p.MB, p.W) + 127) / 128;
    const int64_t table_units = static_cast<int64_t>(p.R) * chunks, units = table_units + (p.max_tokens + 31) / 32;
    const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
    struct Part {  // lane's four entries j0 .. of row r, the pages held there
        int r, j0, v[4];
        bool on;
    };
    auto fetch = [&](int64_t u) {
        Part t;
        t.on = u < table_units;
        if (t.on) {
            t.r = static_cast<int>(table_units <= 0x7fffffff ? static_cast<unsigned>(u) / static_cast<unsigned>(chunks) : u / chunks);
            t.j0 = static_cast<int>(u - static_cast<int64_t>(t.r) * chunks) * 128 + lane * 4;
            const int b0 = blocks(rows[t.r].old_len);
            const int32_t *held = p.pages + static_cast<int64_t>(max(rows[t.r].seq, 0)) * p.MB;
            if (p.vec && t.j0 < b0) {  // (j0 + 3 < MB: rows are whole 16-byte pieces)
                const int4 h = *reinterpret_cast<const int4 *>(held + t.j0);
                t.v[0] = h.x, t.v[1] = h.y, t.v[2] = h.z, t.v[3] = h.w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) t.v[e] = !p.vec && t.j0 + e < b0 ? held[t.j0 + e] : 0;
            }
        }
        return t;
    };
    auto finish = [&](Part &t) {
        if (!t.on) return;
        const int b0 = blocks(rows[t.r].old_len), b1 = blocks(rows[t.r].new_len);
        // (most entries are pages that stay, or lie behind the row's last)
        if (t.j0 + 3 >= min(b0, b1) && t.j0 < max(b0, b1)) {
            const Row row = rows[t.r];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int j = t.j0 + e;
                if (j >= b0 && j < b1) {
                    t.v[e] = p.ring[wrap(first + static_cast<int>(row.taken) + j - b0)];
                    p.pages[static_cast<int64_t>(row.seq) * p.MB + j] = t.v[e];
                } else if (j >= b1) {
                    if (j < b0) p.ring[wrap(wrap(first + count) + static_cast<int>(row.given) + j - b1)] = t.v[e];
                    t.v[e] = 0;
                }
            }
        }
        int32_t *out = p.table + static_cast<int64_t>(t.r) * p.W;
        if (p.vec) {
            if (t.j0 < p.W) *reinterpret_cast<int4 *>(out + t.j0) = make_int4(t.v[0], t.v[1], t.v[2], t.v[3]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (t.j0 + e < p.W) out[t.j0 + e] = t.v[e];
        }
    };
    auto token = [&](int64_t u) {
        const int64_t t = (u - table_units) * 32 + lane;
        if (u < table_units || t >= p.max_tokens) return;
        int64_t slot = -1, pos = 0;
        if (t < total.start) {
            int lo = 0, hi = p.R - 1;  // the last row that starts at t or before: it has tokens
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (rows[mid].start <= static_cast<unsigned>(t)) lo = mid;
                else hi = mid - 1;
            }
            const Row row = rows[lo];
            const int at = row.old_len + static_cast<int>(static_cast<unsigned>(t) - row.start);
            const int j = at >> bs_log2, b0 = blocks(row.old_len);
            const int page = j < b0 ? p.pages[static_cast<int64_t>(row.seq) * p.MB + j]
                                    : p.ring[wrap(first + static_cast<int>(row.taken) + j - b0)];
            pos = at;
            if (page >= 0 && page < p.NB) slot = (static_cast<int64_t>(page) << bs_log2) + (at & bs1);
            else pa::record_error(p.err, PA_DEVERR_BAD_BLOCK);
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    };
    // (CTA by CTA, so that a small step's units lie on different SMs)
    for (int64_t u = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x; u < units; u += AT_ONCE * nwarps) {
        Part t[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) t[k] = fetch(u + k * nwarps);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) finish(t[k]);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) token(u + k * nwarps);
    }
    if (blockIdx.x == 0) {
        for (int i = tid; i < p.R; i += kThreads) {
            p.context_lens[i] = rows[i].new_len;
            p.query_start[i] = static_cast<int>(rows[i].start);
        }
        if (tid == 0) p.query_start[p.R] = static_cast<int>(total.start);
    }

    // (not earlier: CTAs of the next launch that wait beside these cost 1,024 rows a quarter)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // ---- the state advances once every CTA has read it -------------------------------
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        last = gridDim.x == 1 || atomicAdd(&p.state[2], 1) == static_cast<int>(gridDim.x) - 1;
    }
    __syncthreads();
    if (!last) return;
    if (tid == 0) {
        p.state[2] = 0;
        if (why) {
            p.state[3] += 1;
            pa::record_error(p.err, why);
        } else {
            p.state[0] = wrap(first + static_cast<int>(total.taken));
            p.state[1] = count - static_cast<int>(total.taken) + static_cast<int>(total.given);
        }
    }
    if (!why)
        for (int i = tid; i < p.R; i += kThreads)
            if (rows[i].seq >= 0) p.lens[rows[i].seq] = rows[i].new_len;
}

// Validate mode: ids in range and once each, lengths inside the tables, and the
// ring's pages and the sequences' in the pool and once each.
int validate_plan(const PlanParams &p, cudaStream_t stream) try {
    std::vector<int32_t> ids(p.R), lens(p.S), pages(size_t(p.S) * p.MB), ring(p.NB), state(4);
    if (int rc = pa::fetch(ids.data(), p.seq_ids, ids.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(lens.data(), p.lens, lens.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(pages.data(), p.pages, pages.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(ring.data(), p.ring, ring.size() * 4, stream)) return rc;
    if (int rc = pa::fetch(state.data(), p.state, 16, stream)) return rc;
    std::vector<bool> row(p.S), used(p.NB);
    for (int r = 0; r < p.R; ++r) {
        if (ids[r] < 0) continue;
        if (ids[r] >= p.S) return pa::fail(PA_ERR_INVALID, "validate: seq_ids[%d]=%d outside [0,%d)", r, ids[r], p.S);
        if (row[ids[r]]) return pa::fail(PA_ERR_INVALID, "validate: sequence %d is named twice", ids[r]);
        row[ids[r]] = true;
    }
    if (state[0] < 0 || state[0] >= p.NB || state[1] < 0 || state[1] > p.NB || state[2] != 0)
        return pa::fail(PA_ERR_INVALID, "validate: free_state (%d, %d, %d) is no state of %d pages", state[0], state[1],
                        state[2], p.NB);
    auto take = [&](int32_t v) { return v >= 0 && v < p.NB && !used[v] && (used[v] = true); };
    for (int i = 0; i < state[1]; ++i)
        if (!take(ring[(int64_t(state[0]) + i) % p.NB]))
            return pa::fail(PA_ERR_INVALID, "validate: free page %d of the ring is outside the pool or there twice", i);
    for (int s = 0; s < p.S; ++s) {
        const int64_t b = (int64_t(lens[s]) + (1 << p.bs_log2) - 1) >> p.bs_log2;
        if (lens[s] < 0 || b > p.MB)
            return pa::fail(PA_ERR_INVALID, "validate: sequence %d has length %d", s, lens[s]);
        for (int j = 0; j < b; ++j)
            if (!take(pages[size_t(s) * p.MB + j]))
                return pa::fail(PA_ERR_INVALID, "validate: page %d of sequence %d is outside the pool or used twice", j, s);
    }
    return PA_OK;
} catch (const std::bad_alloc &) {
    return pa::fail(PA_ERR_OOM, "validate: host allocation failed");
}

}  // namespace

extern "C" int pa_plan_step(const int32_t *seq_ids, const int32_t *new_tokens, int R, int32_t *seq_pages,
                            int max_blocks_per_seq, int32_t *seq_lens, int num_seqs, int32_t *free_pages,
                            int32_t *free_state, int64_t num_blocks, int block_size, int32_t *block_table,
                            int table_blocks, int32_t *context_lens, int32_t *query_start, int64_t *slots,
                            int64_t *positions, int max_tokens, pa_stream_t stream) {
    pa::clear_error();
    if (R < 0 || num_seqs <= 0 || max_blocks_per_seq <= 0 || table_blocks <= 0 || num_blocks <= 0 || max_tokens < 0)
        return pa::fail(PA_ERR_INVALID, "plan_step: bad sizes");
    if (!pa::pow2_in(block_size, 8, 128))
        return pa::fail(PA_ERR_UNSUPPORTED, "plan_step: block_size %d unsupported", block_size);
    if (R > kMaxRows) return pa::fail(PA_ERR_UNSUPPORTED, "plan_step: %d rows, at most %d", R, kMaxRows);
    if (num_seqs > kMaxSeqs)
        return pa::fail(PA_ERR_UNSUPPORTED, "plan_step: %d sequences, at most %d", num_seqs, kMaxSeqs);
    if (num_blocks > (1 << 30)) return pa::fail(PA_ERR_UNSUPPORTED, "plan_step: more than 2^30 pages");
    if (int64_t(std::max(max_blocks_per_seq, table_blocks)) * block_size > (int64_t(1) << 30))
        return pa::fail(PA_ERR_INVALID, "plan_step: table capacity too large");
    if (max_tokens > (1 << 30)) return pa::fail(PA_ERR_INVALID, "plan_step: max_tokens too large");
    if (!seq_pages || !seq_lens || !free_pages || !free_state || !query_start ||
        (R > 0 && (!seq_ids || !new_tokens || !block_table || !context_lens)) ||
        (max_tokens > 0 && (!slots || !positions)))
        return pa::fail(PA_ERR_INVALID, "plan_step: NULL pointer");
    PlanParams p{};
    p.seq_ids = seq_ids;
    p.change = new_tokens;
    p.pages = seq_pages;
    p.lens = seq_lens;
    p.ring = free_pages;
    p.state = free_state;
    p.table = block_table;
    p.context_lens = context_lens;
    p.query_start = query_start;
    p.slots = slots;
    p.positions = positions;
    p.err = pa::device_error_word();
    p.R = R;
    p.S = num_seqs;
    p.MB = max_blocks_per_seq;
    p.W = table_blocks;
    p.NB = static_cast<int>(num_blocks);
    p.bs_log2 = pa::pf::log2_int(block_size);
    p.max_tokens = max_tokens;
    p.vec = max_blocks_per_seq % 4 == 0 && table_blocks % 4 == 0 && pa::aligned16(seq_pages) &&
            pa::aligned16(block_table);
    if (pa::validate_on())
        if (int rc = validate_plan(p, stream)) return rc;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return pa::cuda_fail(cudaGetLastError(), "plan_step: SM count");
    const size_t smem = size_t(R) * sizeof(Row) + size_t(num_seqs + 31) / 32 * 4;
    static std::atomic<uint64_t> done{0};
    const size_t most = size_t(kMaxRows) * sizeof(Row) + kMaxSeqs / 8;
    if (int rc = pa::pf::set_smem_once(plan_step_kernel, most, &done)) return rc;
    // a unit of each warp, at most a CTA per SM (1,024 rows of 2,048 entries: two CTAs per SM
    // take 10 % longer, four 50 %: each makes all prefix sums)
    const int64_t units = int64_t(R) * ((std::max(p.MB, p.W) + 127) / 128) + max_tokens / 32;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(sms, (units + kWarps - 1) / kWarps))));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    (void)cudaGetLastError();  // drop a stale error that is not ours
    const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_step_kernel, p);
    if (e != cudaSuccess) return pa::cuda_fail(e, "plan_step launch");
    return pa::check_launch("plan_step launch");
}
