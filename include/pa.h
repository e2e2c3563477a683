/*
 * pa.h -- C ABI of the GB300 (sm_103a) paged-attention library.
 *
 * PagedAttention keeps each sequence's KV cache in fixed-size physical blocks
 * and reaches them through a per-sequence block table that maps logical block
 * i to a physical block anywhere in the pool ("PagedAttention: memetakan blok
 * KV logis ke memori fisik tidak kontigu", section "Urutan logis dipisahkan
 * dari penempatan fisik"; "Apa itu PagedAttention?", section "Cara kerja
 * PagedAttention: Blok halaman non-kontigu").  The attention kernel follows
 * the block table before it loads K and V (nalar.dev, section "Kernel
 * attention harus mengikuti block table"); the attention equation itself is
 * unchanged (same page, opening section).
 *
 * Conventions for every call
 * --------------------------
 *  - Return value: PA_OK (0) or a PA_ERR_* code; pa_last_error_string()
 *    gives the message of the last failing call on the calling thread.
 *  - Tensors are caller-owned DEVICE pointers (unless a parameter says host).
 *    The library never allocates device memory in an op call and keeps no
 *    pointer after it returns.
 *  - Ops are asynchronous on the given stream (a cudaStream_t; NULL = the
 *    legacy default stream).  The status covers argument checks and launch
 *    errors only; device-side errors (an out-of-range block id, a pipeline
 *    wait that ran out) are recorded in a device error word read by
 *    pa_device_error().
 *  - dtype: PA_BF16 (bfloat16) or PA_F32 (float32) for q, K/V caches and
 *    outputs.  Accumulation is always fp32.
 *  - Cache layout (both K and V): [num_blocks][Hkv][block_size][head_dim],
 *    contiguous, so one (block, KV head) is block_size*head_dim contiguous
 *    elements.  Pool base pointers must be 16-byte aligned.
 *  - GQA: query head h reads KV head h / (Hq / Hkv).
 *  - Supported shapes: head_dim 64 or 128; Hq/Hkv in {1, 2, 4, 8};
 *    block_size a power of two in [8, 128].
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *pa_stream_t; /* same type as cudaStream_t */

enum {
    PA_OK = 0,
    PA_ERR_INVALID = 1,     /* bad argument, shape or (validate mode) metadata */
    PA_ERR_OOM = 2,         /* block manager: not enough free blocks or host memory */
    PA_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed */
    PA_ERR_UNSUPPORTED = 4, /* valid request this build has no kernel for */
    PA_ERR_DEVICE = 5       /* pa_device_error found a device-side error */
};

enum { PA_BF16 = 0, PA_F32 = 1 };

/* device error word bits (pa_device_error) */
enum {
    PA_DEVERR_BAD_BLOCK = 1, /* a block-table entry was outside [0, num_blocks) */
    PA_DEVERR_TIMEOUT = 2,   /* a bounded pipeline wait ran out; output invalid */
    PA_DEVERR_BAD_REQUEST = 4, /* ids, lengths or rows of a request that do not fit (pa_plan_step,
                                  pa_cross_attention, pa_linear_*) */
    PA_DEVERR_NO_BLOCKS = 8  /* pa_plan_step: the step needs more pages, or a wider table, than there are */
};

/* Message of the last failing call on this thread ("" if none). */
const char *pa_last_error_string(void);

/* Library ABI version (incremented on any signature change). */
int pa_version(void);

/*
 * Validate mode (off by default).  When on, every op first copies its
 * metadata (slot_mapping, block_table, context_lens, copy pairs) to the host
 * and checks it: slots and block ids inside the pool, no duplicate slots in
 * one reshape call, copy pairs disjoint, context lengths in (0, table
 * capacity].  It synchronizes the stream, so it is for debugging and tests.
 */
int pa_set_validate(int on);

/*
 * Read (and, if clear != 0, reset) the device error word of the current
 * device.  Synchronizes the stream.  *bits receives PA_DEVERR_* bits.
 * Returns PA_ERR_DEVICE if any bit was set, else PA_OK.
 */
int pa_device_error(int *bits, int clear, pa_stream_t stream);

/*
 * pa_reshape_and_cache -- store the new tokens' K and V into their slots.
 * Only the new token's K/V is computed and stored; earlier tokens are read
 * back from the cache ("KV Cache dan PagedAttention: Apa Fungsinya dan
 * Mengapa Itu Penting", section "Apa itu KV Cache?").
 *   k_new, v_new  [T][Hkv][head_dim]               (dtype)
 *   k_cache, v_cache  pool as above, written in place
 *   slot_mapping  int64 [T]: slot = physical_block * block_size + offset;
 *                 a negative slot is padding and is skipped
 * Effect: k_cache[slot/bs][h][slot%bs][:] = k_new[t][h][:] (same for V), bit
 * exact.  Duplicate slots in one call are a caller error (undefined which
 * token wins; PA_ERR_INVALID in validate mode).
 */
int pa_reshape_and_cache(const void *k_new, const void *v_new, void *k_cache, void *v_cache,
                         const int64_t *slot_mapping, int64_t T, int64_t num_blocks, int Hkv,
                         int block_size, int head_dim, int dtype, pa_stream_t stream);

/*
 * pa_rope_reshape_and_cache -- pa_reshape_and_cache with rotary positions: the
 * queries and the new keys are rotated by their token's position on the way,
 * in one launch (values are stored as they are).
 * Element pairs (x, y) of a head rotate by the angle a = position * inv_freq[i]
 * of their frequency i in [0, rot_dim/2):
 *   x' = x cos a - y sin a,  y' = x sin a + y cos a
 * with (x, y) = elements (i, i + rot_dim/2), or (2i, 2i + 1) if interleaved;
 * elements from rot_dim on are copied.  A token has one position per axis
 * (one axis for text; time, height and width for images and video); the first
 * sections[0] frequencies take axis 0's position, the next sections[1] axis
 * 1's, and so on.  Angles are taken and reduced in fp64 (off by at most 2^-51 of
 * themselves: 1e-6 at position 2^31); the rotation is fp32, rounded once.
 *   q_out, q      [T][Hq][head_dim], k_new, v_new [T][Hkv][head_dim] (dtype);
 *                 heads of a token contiguous, q_out_stride .. v_stride elements
 *                 (a multiple of 16 bytes, at most 2^28) between tokens: slices
 *                 of one fused projection are fine.  q_out may be q itself, and
 *                 otherwise overlaps no input.
 *   slot_mapping  int64 [T] as for pa_reshape_and_cache (a negative slot stores
 *                 nothing; its query is rotated all the same)
 *   positions     int64 [num_axes][T] device
 *   inv_freq      float32 [rot_dim/2] device
 *   sections      HOST int [num_axes], not negative, summing to rot_dim/2
 *   num_axes      1 .. 4
 * rot_dim: even, at most head_dim and 512, half of it whole 16-byte pieces.
 * head_dim: row of a head a multiple of 16 bytes, at most 1024 elements.
 */
int pa_rope_reshape_and_cache(void *q_out, int64_t q_out_stride, const void *q, int64_t q_stride,
                              const void *k_new, int64_t k_stride, const void *v_new,
                              int64_t v_stride, void *k_cache, void *v_cache,
                              const int64_t *slot_mapping, const int64_t *positions,
                              const float *inv_freq, const int *sections, int num_axes,
                              int interleaved, int64_t T, int64_t num_blocks, int Hq, int Hkv,
                              int block_size, int head_dim, int rot_dim, int dtype,
                              pa_stream_t stream);

/*
 * pa_copy_blocks -- copy-on-write support: for each pair (src, dst), physical
 * block dst of BOTH caches becomes a byte copy of block src ("Apa itu
 * PagedAttention?", section "Cara kerja PagedAttention", item 3; nalar.dev,
 * section "Sharing blok dapat menghindari duplikasi state KV").
 *   pairs  int64 [n][2] device array of (src, dst) block ids
 * No dst may equal any src or another dst in the same call (PA_ERR_INVALID in
 * validate mode).  Bit exact.
 */
int pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *pairs, int64_t n,
                   int64_t num_blocks, int Hkv, int block_size, int head_dim, int dtype,
                   pa_stream_t stream);

/*
 * pa_swap_blocks -- move whole blocks between two pools of the same shape,
 * e.g. swap a sequence's blocks out to pinned host memory and back: when the
 * device pool is full, small pages go to the CPU instead of whole sequences
 * ("KV Cache and PagedAttention: Why Your LLM Server Slows Down", section
 * "How PagedAttention fixes this", fine-grained eviction).
 * For each pair (src, dst): block dst of the destination pools becomes a byte
 * copy of block src of the source pools, K and V.  Each pool (and the pairs
 * array) may be device memory or pinned host memory (reached through its
 * mapped device alias); pageable host memory is rejected.
 *   pairs  int64 [n][2] (src block in the source pool, dst block in the
 *          destination pool); destinations must be distinct (validate mode).
 * Bit exact; asynchronous on the stream like every op.
 */
int pa_swap_blocks(void *dst_k, void *dst_v, const void *src_k, const void *src_v,
                   const int64_t *pairs, int64_t n, int64_t src_num_blocks,
                   int64_t dst_num_blocks, int Hkv, int block_size, int head_dim, int dtype,
                   pa_stream_t stream);

/*
 * pa_compact_cache -- keep some tokens of each sequence and move them to its
 * front: row i of (sequence b, KV head h) becomes the old row keep[b][h][i],
 * K and V, for i < keep_lens[b].  Each KV head keeps tokens of its own; the
 * number kept is the sequence's.  Bit exact.
 *   src_table  int32 [B][src_blocks_per_seq]: the sequences' pages
 *   dst_table  int32 [B][dst_blocks_per_seq]: the pages that receive the kept
 *              tokens.  A page may stay in its place (the same page at the same
 *              logical block of the same sequence: compaction in place); every
 *              other page written must not be read by this call, nor may a page
 *              be written for two sequences.  Pages that other sequences still
 *              share are replaced by fresh ones (pa_bm_compact does this).
 *   keep       int32 [B][Hkv][max_keep] device: strictly ascending positions
 *              inside src_table; entries from keep_lens[b] on are not read
 *   keep_lens  int32 [B], each in [0, max_keep]
 * Validate mode checks every rule above.  Outside it, a position or page out of
 * range is skipped and recorded (PA_DEVERR_BAD_BLOCK); positions that are not
 * ascending, or pages read and written other than in place, give undefined
 * rows.  Rows behind the last kept token keep their old bytes.
 * A row's index is no longer its token's position.  Keys stay rotated by the
 * position that their token had, so the next token's rotary position is still
 * the number of tokens the sequence has had, not its length (the caller counts
 * it); windows and sinks count rows.
 */
int pa_compact_cache(void *k_cache, void *v_cache, const int32_t *src_table,
                     int src_blocks_per_seq, const int32_t *dst_table, int dst_blocks_per_seq,
                     const int32_t *keep, int max_keep, const int32_t *keep_lens, int B,
                     int64_t num_blocks, int Hkv, int block_size, int head_dim, int dtype,
                     pa_stream_t stream);

/*
 * pa_decode_workspace_size -- bytes of device workspace pa_decode needs: the
 * per-item partial counts (4 bytes per (sequence, query head), padded to a
 * multiple of 256 bytes) and the fp32 partials (max, sum and weighted values)
 * of up to partitions-of-the-table-capacity + 1 segments per (sequence,
 * query head).  Non-zero for every B > 0 (0 for B = 0).  partition_tokens as
 * for pa_decode (0 = library default).  PA_ERR_INVALID on bad sizes or when
 * the size does not fit in size_t.
 */
int pa_decode_workspace_size(int B, int Hq, int head_dim, int max_blocks_per_seq,
                             int block_size, int partition_tokens, size_t *bytes);

/* kernels pa_decode can launch (pa_decode_kernel_for) */
enum { PA_DECODE_PERSISTENT = 1, PA_DECODE_GRID = 2 };

/*
 * pa_decode_kernel_for -- which kernel pa_decode launches for a batch of these
 * sizes on the current device.  The choice depends on the sizes only (never
 * on context lengths or device data), so one batch shape always runs the
 * same kernel:
 *   PA_DECODE_PERSISTENT  one persistent grid (2 CTAs of 4 warps per SM) that
 *                         splits the batch's (sequence, KV head, 16-token
 *                         tile) units evenly over its warps;
 *   PA_DECODE_GRID        one CTA per (sequence, KV head, partition), then a
 *                         merge kernel; chosen when B * Hkv * (partitions of
 *                         the table capacity) is at most 1.75 times the
 *                         persistent grid's warp count (little work), and for
 *                         B > 4096.
 * Both meet the same error bound; their results may differ in the last bits
 * (another order of the partial sums).  Arguments as for pa_decode;
 * *kernel receives PA_DECODE_PERSISTENT or PA_DECODE_GRID.  PA_ERR_INVALID
 * on bad sizes, PA_ERR_CUDA without a current device.
 */
int pa_decode_kernel_for(int B, int Hkv, int max_blocks_per_seq, int block_size,
                         int partition_tokens, int *kernel);

/* per-tile math of the persistent decode kernel (pa_decode_tile_for) */
enum { PA_DECODE_TILE_CUDA_CORE = 1, PA_DECODE_TILE_TENSOR_CORE = 2 };

/*
 * pa_decode_tile_for -- how the persistent decode kernel computes a tile of
 * one (sequence, KV head) for these shapes (the grid kernel always uses the
 * CUDA-core tile):
 *   PA_DECODE_TILE_TENSOR_CORE  bf16 with groups of 4 or 8 query heads per KV
 *       head (and num_blocks * Hkv * block_size < 2^31): 16-token tiles by
 *       2D tensor copies (128-byte swizzle); scores and the weighted sum of
 *       values by warp-level bf16 tensor-core MMAs with fp32 accumulation
 *       (the group's heads are the N = 8 columns; softmax weights enter as a
 *       bf16 hi + lo pair);
 *   PA_DECODE_TILE_CUDA_CORE    every other case: packed fp32 FMAs and warp
 *       shuffles.
 * Both meet the same error bound.  PA_ERR_INVALID on bad shapes.
 */
int pa_decode_tile_for(int Hq, int Hkv, int head_dim, int block_size, int64_t num_blocks,
                       int dtype, int *tile);

/*
 * pa_decode -- paged decode attention: one query token per sequence.
 * For sequence b with context length L = context_lens[b] (the newest token,
 * already stored by pa_reshape_and_cache, included) and query head h:
 *   o[b][h] = sum_{j<L} exp(s_j - max s) V_b[j][h/g] / sum_j exp(s_j - max s),
 *   s_j = scale * (q[b][h] . K_b[j][h/g])
 * where token j of sequence b lives in physical block
 * block_table[b][j / block_size] at offset j % block_size.  The sum over j
 * is split into partitions of partition_tokens tokens whose partial
 * (max, sum, weighted values) are merged by log-sum-exp when L exceeds one
 * partition.  The result depends only on the logical token order, never on
 * where blocks sit in the pool (bit-identical under any placement).
 *   out, q        [B][Hq][head_dim]                    (dtype)
 *   block_table   int32 [B][max_blocks_per_seq]
 *   context_lens  int32 [B], each in [1, max_blocks_per_seq*block_size]
 *   partition_tokens  0 = default (512), or a positive multiple of both 32
 *                 and block_size
 *   workspace     device buffer of at least pa_decode_workspace_size bytes,
 *                 16-byte aligned; its contents on entry do not matter (every
 *                 partial and per-item count is written before it is read)
 *                 and it holds scratch afterwards.  Calls that may overlap on
 *                 the GPU need separate workspaces.
 * Launches: the decode grid (persistent or grid kernel, pa_decode_kernel_for)
 * and a kernel that merges the partials of items split across warps or
 * partitions.  Each is launched as a programmatic dependent of the kernel
 * before it in the stream: it may start while that kernel drains, and waits
 * for that kernel to complete before it reads any input.
 */
int pa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
              const int32_t *block_table, int max_blocks_per_seq, const int32_t *context_lens,
              int B, int Hq, int Hkv, int head_dim, int block_size, int64_t num_blocks,
              float scale, int partition_tokens, void *workspace, size_t workspace_bytes,
              int dtype, pa_stream_t stream);

/*
 * pa_decode_contiguous -- the decode of pa_decode over a plain contiguous
 * cache, for measuring what paging costs: each sequence reserves max_len
 * slots up front, the reservation that paging replaces ("Apa itu
 * PagedAttention?", section "Masalah fragmentasi memori KV Cache
 * konvensional"), so no block table is read and no address depends on a
 * table entry.  Following the block table is the cost paging adds
 * ("PagedAttention: memetakan blok KV logis ke memori fisik tidak kontigu",
 * section "Kernel attention harus mengikuti block table").  The kernel is
 * pa_decode's persistent kernel with the same tiles and split; only the
 * address of a tile differs.
 *   k, v   [B][Hkv][max_len][head_dim] device arrays (dtype); token j of
 *          sequence b, KV head h at row (b * Hkv + h) * max_len + j
 *   max_len  a positive multiple of 32; context_lens[b] in [1, max_len]
 *   workspace  at least pa_decode_contiguous_workspace_size bytes
 * Other arguments and the result as for pa_decode.  At most 4096 sequences
 * (PA_ERR_UNSUPPORTED beyond).
 */
int pa_decode_contiguous_workspace_size(int B, int Hq, int head_dim, int max_len,
                                        int partition_tokens, size_t *bytes);
int pa_decode_contiguous(void *out, const void *q, const void *k, const void *v,
                         const int32_t *context_lens, int B, int Hq, int Hkv, int head_dim,
                         int max_len, float scale, int partition_tokens, void *workspace,
                         size_t workspace_bytes, int dtype, pa_stream_t stream);

/*
 * pa_decode_shared -- pa_decode for a batch in which groups of sequences share
 * the physical blocks of a common prefix: a system prompt, or the history of
 * parallel-sampling branches forked from one parent.  A shared block is one
 * physical copy that serves every sequence referencing it ("PagedAttention:
 * memetakan blok KV logis ke memori fisik tidak kontigu", section "Sharing
 * blok dapat menghindari duplikasi state KV"; "Apa itu PagedAttention?",
 * section "Cara kerja PagedAttention", item 3).  Here the shared part is also
 * READ once per (group, KV head): a prefix kernel streams the group's shared
 * blocks once through shared memory and computes the attention partials
 * (max, sum, weighted values) of every member's query heads against them on
 * tensor cores; the decode then covers each member's private tokens only and
 * merges the two parts by log-sum-exp.
 * Same arguments and result as pa_decode (within the same error bound: the
 * sums are taken in another order, so the bits may differ from pa_decode's),
 * plus the groups:
 *   shared_len    int32 [B] device: tokens at the start of sequence b covered by
 *                 its group's shared blocks; a positive multiple of block_size
 *                 below context_lens[b] for a member, 0 for a sequence in no
 *                 group.  All members of a group have the same value and the
 *                 same first shared_len / block_size block-table entries (the
 *                 first member's row is read for the shared blocks).
 *   group_start   int32 [G+1] device: the members of group g are
 *                 group_seqs[group_start[g] .. group_start[g+1]).
 *   group_seqs    int32 [num_members] device: batch rows of the members; a
 *                 sequence belongs to at most one group.
 *   G, num_members, max_group_size, max_shared_len: host ints bounding the
 *                 arrays (max_group_size >= every group's size,
 *                 max_shared_len >= every shared_len).
 *   workspace     at least pa_decode_shared_workspace_size bytes.
 * Validate mode checks every rule above.  Calls that cannot take the shared
 * path (fp32, batches that pa_decode_kernel_for sends to the grid kernel,
 * pools of 2^31 rows or more) decode every sequence whole, which gives the
 * same result.  Launches (each a programmatic dependent of the one before):
 * block sizes 8..64: the decode grid, the tcgen05 prefix kernel (it reads none
 * of the decode's results: the decode grid releases it at its start, so its
 * CTAs take the SMs the decode leaves, and it waits for that grid only before
 * exiting), the merge (released at the prefix kernel's start; it waits for
 * that kernel before it reads anything); other block sizes: the warp-level
 * prefix kernel, the decode grid, the merge.
 * Outside validate mode, a member whose own shared_len is not a positive
 * multiple of block_size below its context length is decoded whole and
 * PA_DEVERR_BAD_BLOCK is recorded; members that disagree with their group's
 * first member (another shared_len or other shared blocks) give undefined
 * output (PA_DEVERR_BAD_BLOCK is recorded for a differing shared_len; other
 * blocks are only caught by validate mode).
 */
int pa_decode_shared_workspace_size(int B, int Hq, int head_dim, int max_blocks_per_seq,
                                    int block_size, int partition_tokens, int max_shared_len,
                                    size_t *bytes);
int pa_decode_shared(void *out, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_table, int max_blocks_per_seq,
                     const int32_t *context_lens, int B, int Hq, int Hkv, int head_dim,
                     int block_size, int64_t num_blocks, float scale, int partition_tokens,
                     const int32_t *shared_len, const int32_t *group_start,
                     const int32_t *group_seqs, int G, int num_members, int max_group_size,
                     int max_shared_len, void *workspace, size_t workspace_bytes, int dtype,
                     pa_stream_t stream);

/*
 * pa_decode_shared_forks -- pa_decode_shared for a batch that also holds
 * forked children ("Apa itu PagedAttention?", section "Cara kerja
 * PagedAttention", item 3: a forked branch shares its parent's blocks until
 * it writes; "PagedAttention: memetakan blok KV logis ke memori fisik tidak
 * kontigu", section "Sharing blok dapat menghindari duplikasi state KV").
 * A child shares with its parent not only the group's prefix but every
 * block before its fork point; here those blocks are read once for both:
 * the parent's K/V tiles over [shared_len, fork_len) also serve the child's
 * query heads (bf16, groups of 4 query heads: the tensor-core tile's spare
 * columns), and the child's own reads start at its fork point.
 * Same arguments and result as pa_decode_shared (within the same error
 * bound), plus:
 *   fork_parent   int32 [B] device: for a child, the batch row of its parent,
 *                 else -1.  A parent is no child itself and has one child.
 *   fork_len      int32 [B] device: for a child, the tokens whose blocks it
 *                 shares with its parent: a positive multiple of block_size
 *                 in [shared_len, both context lengths), the two table rows
 *                 equal before it.  Ignored for other rows.
 *   workspace     at least pa_decode_shared_forks_workspace_size bytes.
 * Validate mode checks every rule above.  Outside it, a child whose fork
 * does not meet them (or the second child of one parent) reads its whole
 * range itself and PA_DEVERR_BAD_BLOCK is recorded; rows that agree on the
 * numbers but not on the blocks give undefined output.  Other shapes (fp32,
 * groups of 1, 2 or 8 heads, the grid kernel) read every range themselves,
 * with the same result.  Launches as pa_decode_shared.  Measured on a fork
 * step of 320 sequences (64 children, ~256 private tokens each): 11 % fewer
 * DRAM reads than pa_decode_shared but 3.4 us slower per call (the fork
 * tile's per-tile masking and wider partial rows cost more than the reads).
 */
int pa_decode_shared_forks_workspace_size(int B, int Hq, int head_dim, int max_blocks_per_seq,
                                          int block_size, int partition_tokens,
                                          int max_shared_len, size_t *bytes);
int pa_decode_shared_forks(void *out, const void *q, const void *k_cache, const void *v_cache,
                           const int32_t *block_table, int max_blocks_per_seq,
                           const int32_t *context_lens, int B, int Hq, int Hkv, int head_dim,
                           int block_size, int64_t num_blocks, float scale, int partition_tokens,
                           const int32_t *shared_len, const int32_t *group_start,
                           const int32_t *group_seqs, int G, int num_members, int max_group_size,
                           int max_shared_len, const int32_t *fork_parent,
                           const int32_t *fork_len, void *workspace, size_t workspace_bytes,
                           int dtype, pa_stream_t stream);

/*
 * pa_decode_noalloc -- pa_decode for callers that cannot allocate device
 * memory (for example a plug-in whose host program owns all device memory
 * through its own pool, or a latency-critical loop where cudaMalloc, which
 * may synchronize the device, is not allowed).  The pages have no
 * counterpart to this entry point; it only changes where the split-KV
 * workspace comes from.
 * Same arguments and result as pa_decode, without workspace: the library
 * uses a fixed device array of pa_decode_noalloc_capacity() bytes (16 MiB)
 * that every GPU loading the library holds until the process exits.  A
 * batch whose pa_decode_workspace_size exceeds it is rejected with
 * PA_ERR_INVALID.  The first call on a device (with that device current)
 * looks up the array's device address; make it before any stream capture.
 * All calls on a device share the array: calls that overlap on the GPU race
 * and must be serialized by the caller.  Nothing is allocated, no
 * cudaMalloc/cudaFree is called.
 */
size_t pa_decode_noalloc_capacity(void);
int pa_decode_noalloc(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_table, int max_blocks_per_seq,
                      const int32_t *context_lens, int B, int Hq, int Hkv, int head_dim,
                      int block_size, int64_t num_blocks, float scale, int partition_tokens,
                      int dtype, pa_stream_t stream);

/*
 * pa_decode_window -- pa_decode with a sliding window and sinks: the new query
 * of sequence b (at position L - 1, L = context_lens[b]) sees the tokens j with
 *   j < num_sinks  or  j >= L - window,
 * the first few of the sequence and the last `window`, the newest included.
 *   window     at least 1; num_sinks at least 0 (both may exceed L)
 *   block_table  entries of blocks that hold no visible token are never read:
 *              their pages may have been freed (pa_bm_trim)
 *   context_lens  each in [0, capacity]; a row of length 0 (padding of a batch)
 *              gets zeros
 * Other arguments and the error bound as for pa_decode; bit-identical under any
 * placement of the blocks.  K and V of tokens that are not visible do not enter
 * the result, whatever they hold.  One launch, without a workspace: a cluster
 * of 1 to 16 CTAs (from the sizes alone) per (sequence, KV head).
 */
int pa_decode_window(void *out, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_table, int max_blocks_per_seq,
                     const int32_t *context_lens, int B, int Hq, int Hkv, int head_dim,
                     int block_size, int64_t num_blocks, float scale, int window, int num_sinks,
                     int dtype, pa_stream_t stream);

/*
 * pa_check_wait_timeout -- diagnostic of the device-side failure path: one
 * warp waits, with the same bounded wait (about 2 s) the pipelined kernels
 * use on their copies and hand-offs, on an mbarrier that nothing completes.
 * The wait runs out, PA_DEVERR_TIMEOUT is recorded in the device error word
 * and the kernel returns: nothing faults and the context stays usable.
 * Asynchronous on `stream`; read the outcome with pa_device_error().
 */
int pa_check_wait_timeout(pa_stream_t stream);

/*
 * pa_prefill_chunk -- chunked prefill over paged context ("Melihat Lebih
 * Dalam vLLM v0.7", section "Blueprint Arsitektur 3: Chunked Prefill": a long
 * prompt is cut into chunks of e.g. 512 tokens and run next to decode).
 * Request r has n_r = query_start[r+1]-query_start[r] new query tokens whose
 * K/V are already in the cache; its context length is L_r = context_lens[r]
 * (prior tokens plus the chunk), so new token i sits at absolute position
 * P_r + i with P_r = L_r - n_r and attends to positions 0..P_r+i (causal).
 *   out, q        [query_start[R]][Hq][head_dim]       (bf16 only)
 *   query_start   int32 [R+1] prefix sum of new-token counts
 *   context_lens  int32 [R]
 *   max_query_len host int >= every n_r (sizes the grid)
 */
int pa_prefill_chunk(void *out, const void *q, const void *k_cache, const void *v_cache,
                     const int32_t *block_table, int max_blocks_per_seq,
                     const int32_t *query_start, const int32_t *context_lens, int R,
                     int max_query_len, int Hq, int Hkv, int head_dim, int block_size,
                     int64_t num_blocks, float scale, int dtype, pa_stream_t stream);

/*
 * pa_prefill_window -- pa_prefill_chunk with a sliding window and sinks: new
 * token i of request r, at position p = P_r + i, sees the tokens j <= p with
 *   j < num_sinks  or  j > p - window.
 *   out, q        [total_tokens][Hq][head_dim]  (bf16 only); rows outside every
 *                 request are left as they are
 *   query_start   int32 [R+1] prefix sum of new-token counts, inside
 *                 [0, total_tokens]; a request may have no new tokens
 *   total_tokens  rows of q and out
 *   max_query_len host int >= every request's new tokens (sizes the grid; with
 *                 less, rows may be left out and PA_DEVERR_BAD_BLOCK recorded)
 *   window        at least 1; num_sinks at least 0 (both may exceed the context)
 *   block_table   entries of blocks that no new token of the request sees are
 *                 never read: their pages may have been freed (pa_bm_trim)
 * Any block size and table length that pa_decode_window takes.  K and V of
 * tokens that no new token of a request sees (slots never written, tokens
 * before the first query's window) do not enter its rows, whatever they hold;
 * a NaN or infinity in V of a token that one of them sees may also reach the
 * rows of the same request and KV head that do not (their weight is 0, and
 * 0 x NaN is NaN).
 * Other arguments and the error bound as for pa_prefill_chunk.  A request whose
 * lengths do not fit (context outside [new tokens, capacity], rows outside
 * [0, total_tokens]) is left out and PA_DEVERR_BAD_BLOCK recorded.  One launch
 * per 256 requests.
 */
int pa_prefill_window(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_table, int max_blocks_per_seq,
                      const int32_t *query_start, const int32_t *context_lens, int R,
                      int total_tokens, int max_query_len, int Hq, int Hkv, int head_dim,
                      int block_size, int64_t num_blocks, float scale, int window, int num_sinks,
                      int dtype, pa_stream_t stream);

/* kernels pa_prefill_window can launch (pa_prefill_window_kernel_for) */
enum { PA_PREFILL_WINDOW_PERSISTENT = 1, PA_PREFILL_WINDOW_SPLIT = 2 };

/*
 * pa_prefill_window_kernel_for -- which kernel pa_prefill_window launches for
 * these sizes on the current device (sizes only, never device data):
 *   PA_PREFILL_WINDOW_SPLIT       a cluster of CTAs per (128 query rows, KV
 *                                 head), when there are at most as many of
 *                                 these as SMs and at most 256 requests;
 *   PA_PREFILL_WINDOW_PERSISTENT  one CTA per SM running a list of (request,
 *                                 256 query rows, KV head) items.
 * Both meet the same error bound.  Arguments as for pa_prefill_window;
 * PA_ERR_INVALID / PA_ERR_UNSUPPORTED on bad sizes, PA_ERR_CUDA without a
 * current device.
 */
int pa_prefill_window_kernel_for(int R, int total_tokens, int max_query_len, int Hq, int Hkv,
                                 int *kernel);

/* kernels pa_prefill_chunk can launch (pa_prefill_kernel_for) */
enum { PA_PREFILL_PERSISTENT_GRID = 1, PA_PREFILL_ITEM_GRID = 2, PA_PREFILL_SIMPLE = 3 };

/*
 * pa_prefill_kernel_for -- which kernel pa_prefill_chunk launches for these
 * sizes (sizes only, never device data; no device needed).  A work item is
 * (request, 256 query rows, KV head).
 *   PA_PREFILL_PERSISTENT_GRID  one CTA per SM (at most one per item), each
 *                               running a list of items dealt longest first
 *                               to the least-loaded CTA; batches of at most
 *                               256 (request, 256-row) pairs and 512 items;
 *   PA_PREFILL_ITEM_GRID        one CTA per item, longest first (larger
 *                               batches);
 *                               both: blocks of 8..64 tokens, tables of at
 *                               most 1024 blocks, fewer than 2^31 pool rows
 *                               of (block, KV head, slot);
 *   PA_PREFILL_SIMPLE           one CTA of 128 threads per 128 rows (every
 *                               other supported size, e.g. 128-token blocks).
 * All three meet the same error bound.  Arguments as for pa_prefill_chunk;
 * *kernel receives the choice.  PA_ERR_INVALID / PA_ERR_UNSUPPORTED as
 * pa_prefill_chunk would return for the sizes.
 */
int pa_prefill_kernel_for(int R, int max_query_len, int Hq, int Hkv, int head_dim,
                          int block_size, int64_t num_blocks, int max_blocks_per_seq,
                          int *kernel);

/*
 * pa_plan_step -- a step's block tables, slots and positions from its requests'
 * lengths, on the device: a captured step (plan, rotary store, attention) needs
 * no host work between two replays.
 * The sequences and their pages live on the device, written by this call only:
 *   seq_pages   int32 [num_seqs][max_blocks_per_seq]: pages of sequence s in
 *               logical order
 *   seq_lens    int32 [num_seqs]: tokens of sequence s (0 at the start)
 *   free_pages  int32 [num_blocks]: a ring of the pages that no sequence holds
 *   free_state  int32 [4]: the ring's first entry, how many there are, a word that
 *               is 0 between calls, and how many steps were refused so far
 *               (at the start: all pages in the ring in any order, 0, num_blocks, 0, 0)
 * A step:
 *   seq_ids     int32 [R]: the sequence of row r, each at most once; negative: a
 *               row of padding (length 0, no tokens)
 *   new_tokens  int32 [R]: c > 0 adds c tokens to the row's sequence, c < 0 drops
 *               its last -c (all of them if it has fewer), as rejected drafts or
 *               a finished request
 * Pages are taken from the ring's front row by row, pages that are no longer
 * needed go behind its end; sequences share no pages.  Out, all of it written and none
 * of it part of the state or the step's inputs:
 *   block_table   int32 [R][table_blocks]: the row's pages, 0 behind them
 *   context_lens  int32 [R]: the new lengths
 *   query_start   int32 [R + 1]: prefix sums of the added tokens
 *   slots         int64 [max_tokens]: slot of each added token, -1 behind the last
 *   positions     int64 [max_tokens]: its position, 0 behind the last
 * slots and positions go by added token, the calls of single tokens (pa_decode_window,
 * pa_linear_decode) by row: the two agree where every row gains one token, or rows that
 * gain none stand behind the others.  In other steps tokens are taken by query_start
 * (pa_prefill_window, pa_cross_attention, pa_linear_prefill).
 * All or nothing: a step that does not fit changes no state, adds no token and
 * shows the old lengths and pages; free_state[3] counts it and PA_DEVERR_NO_BLOCKS
 * (pages, a table too narrow for a row, max_tokens) or PA_DEVERR_BAD_REQUEST (an id
 * past num_seqs or twice, state that this call did not write) is recorded.
 * Validate mode also checks that every page is in the ring or with one sequence.
 * At most 4096 rows and 2^19 sequences; table capacities at most 2^30 tokens.
 * Steps of one state follow one another: calls that may overlap on the GPU, and
 * replays of a graph on two streams, are a caller error.
 */
int pa_plan_step(const int32_t *seq_ids, const int32_t *new_tokens, int R, int32_t *seq_pages,
                 int max_blocks_per_seq, int32_t *seq_lens, int num_seqs, int32_t *free_pages,
                 int32_t *free_state, int64_t num_blocks, int block_size, int32_t *block_table,
                 int table_blocks, int32_t *context_lens, int32_t *query_start, int64_t *slots,
                 int64_t *positions, int max_tokens, pa_stream_t stream);

/*
 * pa_cross_attention -- attention of each request's query tokens to the states of
 * an encoder, kept in pages like any K and V: request r has n_r = query_start[r+1]
 * - query_start[r] query tokens (any number, also none), each of which sees all
 * L_r = encoder_lens[r] states:
 *   o = sum_{j < L_r} softmax(scale q . k_j) v_j;   zeros where L_r = 0
 *   out, q        [total_tokens][Hq][head_dim]  (bf16 only); rows outside every
 *                 request are left as they are
 *   query_start   int32 [R+1] prefix sum of query token counts, inside
 *                 [0, total_tokens]
 *   encoder_lens  int32 [R], each in [0, capacity]
 *   max_query_len host int >= every request's query tokens (with less, rows may be
 *                 left out and PA_DEVERR_BAD_REQUEST recorded); the kernel is chosen by
 *                 it, or by total_tokens where that is less
 * The states of a request are read once for all of its tokens (beams that share an
 * encoder run are the query tokens of one request).  Slots behind the last state
 * do not enter the result, whatever they hold, nor are table entries behind it
 * read; a NaN or infinity in a state reaches the rows of its own request.  A request
 * whose numbers do not fit is left out and PA_DEVERR_BAD_REQUEST recorded.  Other
 * arguments and the error bound as for pa_prefill_window.  At most 65535 requests;
 * one launch per 256 requests, without a workspace.
 */
int pa_cross_attention(void *out, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_table, int max_blocks_per_seq,
                       const int32_t *query_start, const int32_t *encoder_lens, int R,
                       int total_tokens, int max_query_len, int Hq, int Hkv, int head_dim,
                       int block_size, int64_t num_blocks, float scale, int dtype,
                       pa_stream_t stream);

/*
 * pa_linear_decode, pa_linear_decode_planned, pa_linear_prefill -- linear attention
 * with a decay for each head, whose state is all that a sequence keeps:
 *   S_t = l_h S_{t-1} + k_t v_t^T,   o_t = scale * q_t S_t,   l_h = exp(log_decay[h])
 *   out, q, k, v  [tokens][H][head_dim] (dtype); out is contiguous, the others have
 *                 q_stride .. v_stride elements between tokens (heads of a token
 *                 contiguous; a multiple of 16 bytes, at most 2^28); out overlaps
 *                 none of them
 *   states        float32 [num_states][H][head_dim][head_dim], element (i, j) of a
 *                 head belonging to k_i v_j; updated in place
 *   state_ids     int32 [R]: the state of request r, each at most once (a caller
 *                 error otherwise; PA_ERR_INVALID in validate mode)
 *   context_lens  int32 [R]: tokens of the sequence, the new ones included, as
 *                 pa_plan_step gives them.  A request whose context is its new
 *                 tokens alone starts from nothing, whatever its state holds.
 *   log_decay     float32 [H], each at most 0 (a NaN makes the head's outputs and states NaN)
 * pa_linear_decode: one token per request (R = B rows).  A row with a negative
 * state id or context length 0 is padding: zeros, and no state is touched.
 * pa_linear_decode_planned: the same for the rows of a planned step.  query_start,
 * int32 [B + 1], are the step's (NULL: pa_linear_decode).  A row that gained no token
 * (query_start[r + 1] == query_start[r]) is padding too: one that drops tokens or waits,
 * and every row of a step that was refused, which shows the old lengths; without
 * query_start each of them would take a token that its sequence does not have, and a
 * state cannot be taken back.  A row that gained more than one does not fit.  The token
 * of row r is row r of q, k and v, so that a plan's slots, which go by added token, are
 * those of the rows only if rows without a token stand behind the others
 * (pa_linear_prefill with max_query_len 1 takes tokens by query_start, at the same cost).
 * Tokens that a plan drops are not taken out of a state: keep a copy of it before drafts.
 * pa_linear_prefill: request r has the rows query_start[r] .. query_start[r + 1]
 * of total_tokens; a request without new tokens, or with a negative state id, is
 * left out, and rows outside every request are left as they are.  max_query_len
 * >= every request's new tokens; the kernel is chosen by it (or by total_tokens where that
 * is less), so a bound far above the lengths costs time: 64 requests of one token, 32
 * heads of 128, take 43 us with 1 and 105 with 2048.
 *   workspace     device buffer of at least pa_linear_prefill_workspace_size
 *                 bytes, 16-byte aligned, scratch (may be NULL if that is 0);
 *                 calls that may overlap on the GPU need separate ones
 * A request whose numbers do not fit is left out (of a decode: zeros) and
 * PA_DEVERR_BAD_REQUEST recorded.  Sums and states are kept in fp32.  fp32 prompts run
 * token by token on the decode's kernel, as do bf16 prompts of few tokens.  Others run in
 * chunks of 64 tokens, where what is not finite reaches more than the formula says:
 *   - a NaN or infinity in v of a token may also make earlier outputs of the same
 *     request and head within 64 tokens of it NaN (their weight for it is 0, and 0 x NaN
 *     is NaN); one in q or k reaches no earlier token;
 *   - an infinity in q, k or v may come out as NaN where the formula has an infinity.  An
 *     infinite state stays infinite, and v's infinities reach the state as such, as long
 *     as the decays between are not 0 in fp32.
 */
int pa_linear_decode(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                     const void *v, int64_t v_stride, float *states, int num_states,
                     const int32_t *state_ids, const int32_t *context_lens, const float *log_decay,
                     int B, int H, int head_dim, float scale, int dtype, pa_stream_t stream);
int pa_linear_decode_planned(void *out, const void *q, int64_t q_stride, const void *k,
                             int64_t k_stride, const void *v, int64_t v_stride, float *states,
                             int num_states, const int32_t *state_ids, const int32_t *query_start,
                             const int32_t *context_lens, const float *log_decay, int B, int H,
                             int head_dim, float scale, int dtype, pa_stream_t stream);
int pa_linear_prefill_workspace_size(int R, int total_tokens, int max_query_len, int H, int head_dim,
                                     int dtype, size_t *bytes);
int pa_linear_prefill(void *out, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                      const void *v, int64_t v_stride, float *states, int num_states,
                      const int32_t *state_ids, const int32_t *query_start,
                      const int32_t *context_lens, const float *log_decay, int R, int total_tokens,
                      int max_query_len, int H, int head_dim, float scale, void *workspace,
                      size_t workspace_bytes, int dtype, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * Host block manager (opaque handle; C++ behind the C ABI).
 *
 * Free list, per-block reference counts, sequences as lists of physical
 * blocks, fork (prefix sharing), append with copy-on-write.  A new block is
 * taken only when a sequence crosses a block boundary ("Melihat Lebih Dalam
 * vLLM v0.7", section "Blueprint Arsitektur 2", item "Alokasi On-Demand");
 * shared blocks stay shared while unchanged and the branch that writes into a
 * shared, partly filled last block gets a copy first (copy-on-write).  A full
 * shared block needs no copy.  Sharing is explicit (fork), never by content.
 *
 * Free-list order: a stack; initially 0..num_blocks-1, or a Fisher-Yates
 * shuffle driven by SplitMix64(seed) when seed != 0; allocation takes the next
 * block of that order and freed blocks are reused first.
 * Every failing call leaves the manager unchanged.  Not thread safe.
 * ---------------------------------------------------------------------- */
typedef struct pa_bm pa_bm;

int pa_bm_create(int64_t num_blocks, int block_size, uint64_t seed, pa_bm **out);
void pa_bm_destroy(pa_bm *bm);

/* New sequence seq holding n_tokens prompt tokens; slots (host int64
 * [n_tokens], may be NULL) receives their slots.  PA_ERR_INVALID if seq
 * exists, PA_ERR_OOM if too few free blocks. */
int pa_bm_add_seq(pa_bm *bm, int64_t seq, int64_t n_tokens, int64_t *slots);

/* child shares all of parent's blocks (refcount + 1 each). */
int pa_bm_fork(pa_bm *bm, int64_t parent, int64_t child);

/* One new token for seq: *slot receives its slot; (*cow_src, *cow_dst) the
 * block copy to run before writing it, or (-1, -1). */
int pa_bm_append(pa_bm *bm, int64_t seq, int64_t *slot, int64_t *cow_src, int64_t *cow_dst);

/* n new tokens (host int64 slots[n]); at most one copy-on-write pair (only
 * the first new token can hit a shared block). */
int pa_bm_append_n(pa_bm *bm, int64_t seq, int64_t n, int64_t *slots, int64_t *cow_src,
                   int64_t *cow_dst);

/* Drop seq; blocks whose refcount reaches 0 return to the free list. */
int pa_bm_free_seq(pa_bm *bm, int64_t seq);

/* Free the blocks of seq that a sliding window has left: those whose tokens
 * are all in [num_sinks, len - window), which neither the newest token nor any
 * later one sees (pa_decode_window, pa_prefill_window).  Their places in the
 * block list and table become -1; *freed (may be NULL) receives how many the
 * sequence gave up (a shared block returns to the free list with its last
 * holder).  Calls that read the whole context (pa_decode and the like) no longer
 * work on the sequence.  The first queries of a chunk see farther back than the
 * newest token: trim before a chunk is appended or after it has been computed. */
int pa_bm_trim(pa_bm *bm, int64_t seq, int64_t window, int64_t num_sinks, int64_t *freed);

/* Block lists for a compaction (pa_compact_cache) of n sequences to n_tokens[i]
 * tokens each (at most their length): a block that the sequence alone holds
 * stays at its logical place, a shared one, or the place of one that pa_bm_trim
 * gave up, gets a fresh block, and the blocks past the kept tokens are dropped.  Take the sequences'
 * block tables before (src_table) and after (dst_table), and launch the
 * compaction before anything else writes into blocks given out later.
 * pa_bm_seq_len counts the kept rows from here on: it is not the next token's
 * rotary position.  All or nothing; PA_ERR_OOM when there are too few free
 * blocks. */
int pa_bm_compact(pa_bm *bm, const int64_t *seqs, int n, const int64_t *n_tokens);

/* Host int32 out[n][max_blocks]: the block table rows of seqs[0..n), padded
 * with 0 (-1 where pa_bm_trim freed a block).  PA_ERR_INVALID if a sequence is
 * unknown or has more blocks. */
int pa_bm_block_table(const pa_bm *bm, const int64_t *seqs, int n, int32_t *out,
                      int max_blocks);

int pa_bm_seq_len(const pa_bm *bm, int64_t seq, int64_t *len);
/* Physical blocks of seq in logical order: out[cap], *n = number of blocks. */
int pa_bm_seq_blocks(const pa_bm *bm, int64_t seq, int32_t *out, int64_t cap, int64_t *n);
int pa_bm_refcount(const pa_bm *bm, int64_t block, int *refcount);
int64_t pa_bm_num_free(const pa_bm *bm);

/*
 * Host fault injection, for tests of the failure path: from now on the k-th
 * point at which a block-manager call may allocate host memory (k = 0: the
 * next one) fails as if memory had run out; the call returns PA_ERR_OOM and
 * leaves the manager unchanged.  One failure per arming; k < 0 disarms.
 * Process-wide, not thread safe; never armed unless a caller arms it.
 */
void pa_bm_inject_alloc_failure(int64_t k);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
