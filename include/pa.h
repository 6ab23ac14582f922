/*
 * pa.h - C ABI of the GB300 (sm_103a) paged-KV attention library (libpa.so).
 *
 * The KV cache is a pool of fixed-size physical blocks of 16 tokens (or 32, 64 or 128
 * through the *_bs entry points) placed anywhere in device memory; a sequence reaches its blocks through a block table that maps logical
 * block i to a physical block id ("vLLM Internals: From PagedAttention to Removing
 * PagedAttention", section 1.1; "My Understanding of vLLM and PagedAttention", sections
 * "Logical Blocks", "Physical Blocks" and "Block Table"). The table is a dense int32
 * array [num_seqs][max_blocks_per_seq] and new tokens reach the pool through an int64
 * slot mapping ("vLLM: what PagedAttention turned into", section "The problem
 * PagedAttention was actually solving"). Block id 0 is the null block: an ordinary block
 * that "no block" points at, so that padding needs no sentinel ("vLLM: what
 * PagedAttention turned into", section "The block pool").
 *
 * Layouts (all row-major, all device memory, element type given by pa_dtype; BS is the
 * block size, 16 for the plain entry points and the block_size argument of the *_bs ones):
 *   k_cache, v_cache   [num_blocks][num_kv_heads][BS][head_dim]  (one (block, head) page
 *                      of BS x head_dim elements is contiguous)
 *   slot               physical_block * BS + offset_in_block; position p of a sequence
 *                      lives in logical block p / BS at offset p % BS (0-based)
 *   q, out (decode)    [num_seqs][num_q_heads][head_dim]
 *   q, out (prefill)   [total_query_tokens][num_q_heads][head_dim], sequences packed in
 *                      the order of query_start_loc
 *   GQA                query head h reads kv head h / (num_q_heads / num_kv_heads)
 *
 * Conventions shared by every entry point:
 *   - Every pointer is a device pointer owned and allocated by the caller (the block
 *     manager's calls, which take host arrays, excepted); the library allocates no device
 *     memory at run time and keeps no per-call state. Per device it holds the error word, the
 *     fixed scratch of pa_decode_noalloc, and pa_step's side stream and two events. Device
 *     pointers must be 16-byte aligned unless an entry point states otherwise.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL = legacy
 *     default stream). They never read device data on the host and never synchronise
 *     (pa_get_device_errors excepted).
 *   - Arguments that the host can check (null pointers, sizes, head ratio, head_dim,
 *     dtype, workspace size, alignment) are checked before anything is launched; a bad
 *     one returns PA_ERR_INVALID_ARG or PA_ERR_UNSUPPORTED and launches nothing.
 *     A failed launch returns PA_ERR_CUDA.
 *   - Device data that the host cannot check (slots, block ids, lengths) is range-checked
 *     by the kernels: an out-of-range slot is not written, an out-of-range block id or a
 *     length beyond max_blocks_per_seq * BS is not read; each sets a bit in the device
 *     error word (pa_get_device_errors). Kernels never trap.
 *   - seq_lens[i] counts every key of sequence i, the current token(s) included.
 *   - Only the first ceil(seq_lens[i] / BS) entries of block-table row i are read; the
 *     unused tail of a sequence's last block is never read into a result (its contents
 *     may be anything, NaN included), nor is block 0 unless a table names it.
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PA_BLOCK_SIZE 16

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

typedef enum {
    PA_OK = 0,
    PA_ERR_INVALID_ARG = 1,   /* a host-checkable argument is wrong; nothing launched  */
    PA_ERR_UNSUPPORTED = 2,   /* valid but not implemented (e.g. head_dim 96)           */
    PA_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed                   */
    PA_ERR_NO_SPACE = 4       /* block manager: not enough free blocks (nothing changed),
                                 or an output array too small for the answer            */
} pa_status;

typedef enum {
    PA_F32 = 0,               /* fp32 Q/K/V/out, fp32 arithmetic (no TF32)              */
    PA_BF16 = 1,              /* bf16 Q/K/V/out, fp32 accumulation                      */
    PA_FP4 = 2                /* a pool held in 4 bits ("4-bit pools" below): accepted only
                                 where an entry point says so                           */
} pa_dtype;

/* Bits of the device error word. */
#define PA_DEVERR_SLOT_RANGE   0x1u  /* reshape_and_cache met a slot >= num_blocks * BS   */
#define PA_DEVERR_BLOCK_RANGE  0x2u  /* a block-table entry outside [0, num_blocks)       */
#define PA_DEVERR_LEN_RANGE    0x4u  /* a length beyond the table row or max_seq_len      */
#define PA_DEVERR_WAIT_TIMEOUT 0x8u  /* a bounded pipeline wait gave up (results invalid) */
#define PA_DEVERR_APPEND_SLOT  0x10u /* pa_decode_append: slot_mapping[i] is not the slot the
                                        block table gives position seq_lens[i] - 1          */
#define PA_DEVERR_PREFIX_MISMATCH 0x20u /* pa_decode_shared_prefix: a table row does not start
                                           with row 0's prefix blocks (results invalid)   */
#define PA_DEVERR_PAIR_ORDER   0x40u /* pa_move_blocks: src ids not strictly ascending while a
                                        block table is rewritten (the table is unspecified)  */
#define PA_DEVERR_POSITION     0x80u /* pa_rotate_and_cache: a position outside the table of angles (the
                                        token is left out)                                   */

/*
 * pa_reshape_and_cache: write the K/V rows of num_tokens new tokens into their slots.
 * For token t with s = slot_mapping[t] >= 0, and every kv head h:
 *   k_cache[s / 16][h][s % 16][:] = k[t][h][:]   and the same for v.
 * The copy is bitwise in the stored type. A negative slot means "no write" (padding may
 * use either a negative slot or a slot inside null block 0). Slots must be distinct
 * unless they point into block 0 (duplicate non-null slots give an unspecified winner).
 *
 *   k, v          [num_tokens][num_kv_heads][head_dim]   (read)
 *   k_cache       [num_blocks][num_kv_heads][16][head_dim] (written at the slots)
 *   slot_mapping  [num_tokens] int64                       (read)
 * Source: "vLLM: what PagedAttention turned into", section "The problem PagedAttention
 * was actually solving" (int64 slot_mapping); "My Understanding of vLLM and
 * PagedAttention", "Step 3 - Tokens Generated Sequentially" (new K/V are added to the
 * cache as tokens are produced).
 */
PA_API pa_status pa_reshape_and_cache(const void* k, const void* v, void* k_cache, void* v_cache,
                               const int64_t* slot_mapping, int32_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                               pa_dtype dtype, void* stream);

/*
 * Block-size variants. The page "vLLM: what PagedAttention turned into" (intro table and
 * "The problem PagedAttention was actually solving") gives 16 tokens as the block size and
 * reports sizes from 16 to 128 performing alike. Each *_bs entry point is its plain
 * counterpart with the block size as an argument: block_size must be 16, 32, 64 or 128
 * (another positive value returns PA_ERR_UNSUPPORTED, zero or a negative one
 * PA_ERR_INVALID_ARG), and every "16" of the plain entry point's description (pool layout,
 * slot arithmetic, table reads, length bound) reads block_size. The kernels walk a block
 * as block_size / 16 consecutive 16-token pages, so results are bit-identical to the same
 * keys stored in 16-token blocks. pa_decode_workspace_size does not depend on the block size.
 */
PA_API pa_status pa_reshape_and_cache_bs(const void* k, const void* v, void* k_cache, void* v_cache,
                                         const int64_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                                         int32_t head_dim, int32_t num_blocks, int32_t block_size, pa_dtype dtype,
                                         void* stream);

/*
 * pa_decode_workspace_size: bytes of device scratch that pa_decode needs for this shape on
 * the current device (split-KV partial results; on the bf16 path for groups of 4..16 q heads
 * per kv head, also one merge counter per (sequence, kv head) at its start). The caller
 * allocates it and zero-fills it once before its first use. On that bf16 path every call
 * that completes without a device error puts the counters back to zero, so the same buffer
 * serves any number of later calls (and CUDA-graph replays) without re-initialisation. The
 * general path (fp32, or fewer than 4 q heads per kv head) writes plain partial results over
 * the whole buffer: zero-fill it again before a bf16 grouped call reuses a buffer that the
 * general path used, and after a call that raised PA_DEVERR_WAIT_TIMEOUT. Calls that use the
 * same workspace must not overlap on the GPU.
 */
PA_API size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t max_seq_len, pa_dtype dtype);

/*
 * pa_decode: one query row per sequence, at position seq_lens[i] - 1, attending to keys
 * 0..seq_lens[i]-1 gathered through block_table row i inside the kernel:
 *   out[i][h] = softmax_j(scale * q[i][h] . K_i[j]) V_i[j],  K_i[j] = k_cache[bt[i][j/16]][h/G][j%16]
 * A sequence with seq_lens[i] == 0 gets an all-zero output row.
 * Long sequences are split into pieces whose (max, sum, partial output) are merged with a
 * log-sum-exp reduce: on the bf16 path (GQA groups of 4..16) by the last warp to finish a
 * piece of each (sequence, kv head), inside the same kernel; on the general path by a
 * separate reduce kernel. Everything launches on `stream`.
 *
 *   out            [num_seqs][num_q_heads][head_dim]           (written)
 *   q              [num_seqs][num_q_heads][head_dim]           (read)
 *   block_table    [num_seqs][max_blocks_per_seq] int32         (read)
 *   seq_lens       [num_seqs] int32, each in [0, max_seq_len]   (read)
 *   max_seq_len    host-side upper bound of seq_lens (the host never reads seq_lens)
 *   scale          logit scale, usually 1/sqrt(head_dim)
 *   workspace      >= pa_decode_workspace_size(...) bytes of device scratch, 16-B aligned,
 *                  zero-filled before its first use (see pa_decode_workspace_size)
 * Supported: head_dim 64 or 128; num_q_heads % num_kv_heads == 0; bf16 or fp32.
 * Source: "My Understanding of vLLM and PagedAttention", sections "PagedAttention CUDA
 * Kernel" and "Step 4 - Attention Computation" (gather scattered blocks, restore logical
 * order, compute attention); "vLLM Internals", section 4.1 (block tables read inside the
 * attention kernel).
 */
PA_API pa_status pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache,
                    const int32_t* block_table, int32_t max_blocks_per_seq,
                    const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                    int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                    int32_t num_blocks, float scale, pa_dtype dtype,
                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * pa_decode_shared_prefix: pa_decode for a batch whose sequences all begin with the same
 * prefix_tokens keys in the same physical blocks (the first prefix_tokens / 16 entries of every
 * block-table row equal row 0's). Identical prefixes point at the same physical blocks
 * ("vLLM Internals", section 1.2); this call also computes over them once instead of once per
 * sequence. The result is pa_decode's (same arguments, bf16 only), up to rounding: softmax over
 * a sequence's keys is split into the shared prefix and the sequence's own suffix, each reduced
 * to (normalised output, max, sum), and the two are merged by the log-sum-exp rule.
 *   - The suffix part is the balanced decode kernel over keys [prefix_tokens, seq_lens[i]),
 *     on a grid capped to leave SMs for the prefix part, written as fp32 parts into the
 *     workspace; it also checks the table: a row whose prefix entries differ from row 0's sets
 *     PA_DEVERR_PREFIX_MISMATCH (the results are then invalid). The prefix part runs on the
 *     tensor cores, all sequences' query rows of one kv head together against the prefix's key
 *     tiles (no causal bound), as a programmatic dependent launch: it starts on the free SMs
 *     while the decode streams, waits for the decode grid only at its end, merges each row's
 *     suffix part and writes `out`. Both kernels launch on `stream`.
 *   - prefix_tokens: a positive multiple of 16, at most max_seq_len; every seq_lens[i] must be
 *     at least prefix_tokens (a shorter one sets PA_DEVERR_LEN_RANGE).
 *   - Supported: bf16, head_dim 128, 4, 8 or 16 q heads per kv head, at most 1024 sequences
 *     (PA_ERR_UNSUPPORTED otherwise).
 *   - workspace: >= pa_decode_shared_prefix_workspace_size(...) bytes, 16-byte aligned,
 *     zero-filled before its first use, under the rules of pa_decode_workspace_size (its first
 *     part is the suffix decode's workspace).
 *   - flags: 0, or the promises PA_DECODE_TABLES_READY / PA_DECODE_POOL_READY of
 *     pa_decode_append (below) about the kernel launched just before this call; with
 *     POOL_READY that kernel writes no pool row of keys 0 .. seq_lens[i] - 1. They let the
 *     suffix decode scan the lengths and start its first page copies before its wait.
 *     Other bits: PA_ERR_INVALID_ARG.
 * No counterpart entry point exists on the source pages; they describe the sharing of the
 * blocks, and this computes on that sharing.
 */
PA_API size_t pa_decode_shared_prefix_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                                     int32_t head_dim, int32_t max_seq_len, int32_t prefix_tokens);
PA_API pa_status pa_decode_shared_prefix(void* out, const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_table, int32_t max_blocks_per_seq,
                                         const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                                         int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                         int32_t num_blocks, float scale, int32_t prefix_tokens, void* workspace,
                                         size_t workspace_bytes, uint32_t flags, void* stream);

/*
 * pa_decode_append: one decode step with its new tokens, in one launch where it can be. For
 * each sequence i the token at position seq_lens[i] - 1 is new: its K and V rows k_new[i],
 * v_new[i] ([num_seqs][num_kv_heads][head_dim]) are written to slot slot_mapping[i] of the
 * pool, exactly as pa_reshape_and_cache_bs writes them, and decode attention runs over keys
 * 0 .. seq_lens[i] - 1 as pa_decode_bs does. New K/V reach the cache as each token is produced
 * ("My Understanding of vLLM and PagedAttention", "Step 3 - Tokens Generated Sequentially");
 * fusing the write into the attention launch is this library's, not the pages'.
 *
 * On the bf16 persistent path (GQA groups 4..16) one kernel does both: attention takes the new
 * rows from k_new / v_new, so it never waits for its own pool writes. Elsewhere the call
 * launches pa_reshape_and_cache's kernel and then the decode kernel. Either way the results
 * equal pa_reshape_and_cache_bs followed by pa_decode_bs when slot_mapping[i] is the slot that
 * block-table row i gives position seq_lens[i] - 1; on the fused path a slot that is not (a
 * negative one included) sets PA_DEVERR_APPEND_SLOT, the write still goes to slot_mapping[i]
 * (skipped if negative) and attention uses the new rows at position seq_lens[i] - 1.
 * Arguments as for pa_decode_bs, plus k_new, v_new (16-byte aligned) and slot_mapping
 * (int64 [num_seqs], 8-byte aligned); workspace as for pa_decode.
 *
 * flags: 0, or an OR of the bits below; any other bit returns PA_ERR_INVALID_ARG. The fused
 * kernel is a programmatic launch: it may start while the kernel launched just before it on
 * `stream` still runs, and it waits for that kernel to complete before it reads what the flags
 * do not declare ready. It lets the next kernel start only after that wait, so every kernel
 * before the previous one has completed when it starts.
 *   PA_DECODE_TABLES_READY: the kernel launched just before this call writes neither seq_lens
 *     nor block_table (they come from host copies or an earlier step). The kernel then scans
 *     the lengths and loads its first block ids before the wait; the pool, the queries, the
 *     new rows, the output and the workspace are touched after it.
 *   PA_DECODE_POOL_READY (implies PA_DECODE_TABLES_READY): in addition, that kernel writes no
 *     pool row this call reads (keys 0 .. seq_lens[i] - 2; this call writes the new rows
 *     itself). In a model's decode step the kernel before attention produces q, k_new and
 *     v_new, never the pool, so the promise holds there. The kernel then also starts its first
 *     page copies before the wait; the queries, the new rows, the output and the workspace are
 *     still touched after it.
 */
#define PA_DECODE_TABLES_READY 1u
#define PA_DECODE_POOL_READY 2u

PA_API pa_status pa_decode_append(void* out, const void* q, const void* k_new, const void* v_new,
                                  const int64_t* slot_mapping, void* k_cache, void* v_cache,
                                  const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                  int32_t num_seqs, int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t num_blocks, int32_t block_size, float scale,
                                  pa_dtype dtype, void* workspace, size_t workspace_bytes, uint32_t flags,
                                  void* stream);

/* pa_decode with block_size (see the block-size variants above). */
PA_API pa_status pa_decode_bs(void* out, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                              int32_t num_seqs, int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                              int32_t head_dim, int32_t num_blocks, int32_t block_size, float scale, pa_dtype dtype,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * pa_prefill_chunk: causal attention for a chunk of new query tokens per sequence, on top
 * of the sequence's earlier context already in the pool (chunked prefill: a long prompt is
 * processed in pieces interleaved with decode, "vLLM Internals", section 2; a chunk is
 * whatever the token budget leaves, "vLLM: what PagedAttention turned into", section "The
 * scheduler"). Chunk rows are bottom-right aligned: sequence i has
 * C_i = query_start_loc[i+1] - query_start_loc[i] query rows; row r sits at position
 * seq_lens[i] - C_i + r and attends to keys 0..seq_lens[i] - C_i + r. The chunk's own K/V
 * must already be in the pool (pa_reshape_and_cache first).
 *
 *   out, q          [query_start_loc[num_seqs]][num_q_heads][head_dim]
 *   block_table     [num_seqs][max_blocks_per_seq] int32
 *   seq_lens        [num_seqs] int32, total keys incl. this chunk, <= max_seq_len
 *   query_start_loc [num_seqs + 1] int32 prefix sums of chunk lengths (starts at 0),
 *                   every chunk length in [0, min(seq_lens[i], max_chunk_len)]
 * Supported: bf16, head_dim 128 (tensor-core path) and the general CUDA-core path for
 * head_dim 64/128 in bf16 or fp32.
 */
PA_API pa_status pa_prefill_chunk(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_table, int32_t max_blocks_per_seq,
                           const int32_t* seq_lens, const int32_t* query_start_loc,
                           int32_t num_seqs, int32_t max_chunk_len, int32_t max_seq_len,
                           int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t num_blocks, float scale, pa_dtype dtype, void* stream);

/* pa_prefill_chunk with block_size (see the block-size variants above). */
PA_API pa_status pa_prefill_chunk_bs(void* out, const void* q, const void* k_cache, const void* v_cache,
                                     const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                     const int32_t* query_start_loc, int32_t num_seqs, int32_t max_chunk_len,
                                     int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t num_blocks, int32_t block_size, float scale,
                                     pa_dtype dtype, void* stream);

/*
 * pa_decode_noalloc: pa_decode for callers that cannot allocate device memory. The source
 * pages have no counterpart for this entry point; it exists for callers such as a host
 * framework that owns the whole device-memory budget and lets no plug-in allocate, a plug-in
 * that only receives tensors and has no allocator, or a latency-critical path that must not
 * call cudaMalloc/cudaFree (they can synchronise the device).
 *
 * Same arguments and results as pa_decode, without the workspace: the split-KV scratch lives
 * in a fixed array of PA_DECODE_NOALLOC_MAX_BYTES that the library holds in device memory on
 * every GPU that loads it, until the process exits. The call allocates nothing (no
 * cudaMalloc, cudaFree or allocating library routine).
 *   - Shapes whose pa_decode_workspace_size exceeds PA_DECODE_NOALLOC_MAX_BYTES are rejected
 *     with PA_ERR_UNSUPPORTED before anything is launched.
 *   - The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 *     with that device current; make that first call before any stream capture.
 *   - Every call shares the one array, which keeps what the previous call left; the call
 *     itself clears the part that must start at zero (an asynchronous memset on `stream`).
 *     Calls that overlap on the GPU (different streams, or concurrent graphs) race on the
 *     array and give wrong results: serialise them.
 */
#define PA_DECODE_NOALLOC_MAX_BYTES (16u * 1024u * 1024u)

PA_API pa_status pa_decode_noalloc(void* out, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_table, int32_t max_blocks_per_seq,
                                   const int32_t* seq_lens, int32_t num_seqs, int32_t max_seq_len,
                                   int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                   int32_t num_blocks, float scale, pa_dtype dtype, void* stream);

/*
 * pa_step: one whole mixed step of the serving loop in one call: write the step's new K/V
 * into the pool, then chunked-prefill attention for the prefill sequences and decode
 * attention for the decode sequences, with the two attention kernels running side by side.
 * The pages make the per-step work a fixed launch sequence with no host round trip ("vLLM:
 * what PagedAttention turned into", "The scheduler" and the model-runner rewrite: persistent
 * buffers and captured graphs remove per-step CPU work); a step mixes prefill chunks with
 * decode tokens ("vLLM Internals", section 2, chunked prefill).
 *
 * Results are those of the three separate calls (pa_reshape_and_cache_bs, then
 * pa_prefill_chunk_bs and pa_decode_bs on the same pool). Decode is bound by HBM and
 * prefill by the tensor cores, so when both are present and decode takes the bf16
 * persistent path, the decode kernel is given decode_sms SMs and prefill runs on the others
 * at the same time:
 *   stream:  reshape_and_cache -> decode (decode_sms persistent CTAs) -> [join]
 *   side:                     +-> prefill ---------------------------+
 * The side stream and two fork/join events are the library's own, one set per device,
 * created by the first call on that device (make it before any stream capture); the
 * fork/join goes through them under a lock, so pa_step is capturable into a CUDA graph
 * (the side stream joins the capture) and calls from several threads serialise their
 * prefills on the one side stream. Otherwise (no prefill, no decode, or a decode shape that
 * takes the general path) the kernels run one after another on `stream`.
 *
 * A part with zero sequences (or zero new tokens) is skipped and its pointers may be NULL.
 * Every argument is checked as the separate entry point would check it before anything is
 * launched. decode_sms: 0 = 27/64 of the device's SMs (64 of 152, the best split measured for
 * a step of 2 GB of decode KV beside 16 x 512-token prefill chunks); otherwise 1..num_SMs
 * (larger values are clamped). On a capped grid the decode kernel runs 10 warps per CTA.
 * workspace: >= pa_decode_workspace_size(num_decode_seqs, ...) bytes, as for
 * pa_decode. timing_events: NULL, or six cudaEvent_t (each may be NULL) recorded before and
 * after reshape_and_cache, prefill and decode on the stream each kernel runs on, for the
 * caller's profiling; they are recorded as external events, so under stream capture they
 * become event-record nodes of the graph (an event between two kernels stops the later one
 * from launching early).
 */
typedef struct {
    /* the pool and the attention shape shared by every part */
    void* k_cache;
    void* v_cache;
    int32_t num_blocks, block_size;            /* block_size: 16, 32, 64 or 128           */
    int32_t num_q_heads, num_kv_heads, head_dim;
    float scale;
    pa_dtype dtype;
    /* new tokens of the step (pa_reshape_and_cache) */
    const void* k_new;
    const void* v_new;
    const int64_t* slot_mapping;
    int32_t num_new_tokens;
    /* chunked-prefill part (pa_prefill_chunk) */
    void* prefill_out;
    const void* prefill_q;
    const int32_t* prefill_block_table;
    int32_t prefill_max_blocks_per_seq;
    const int32_t* prefill_seq_lens;
    const int32_t* query_start_loc;
    int32_t num_prefill_seqs, max_chunk_len, prefill_max_seq_len;
    /* decode part (pa_decode) */
    void* decode_out;
    const void* decode_q;
    const int32_t* decode_block_table;
    int32_t decode_max_blocks_per_seq;
    const int32_t* decode_seq_lens;
    int32_t num_decode_seqs, decode_max_seq_len;
    void* workspace;
    size_t workspace_bytes;
    /* scheduling */
    int32_t decode_sms;
    void* const* timing_events;
} pa_step_desc;

PA_API pa_status pa_step(const pa_step_desc* step, void* stream);

/*
 * Scored attention: decode and chunked prefill over the paged pool with scores that are capped,
 * biased by distance or masked beyond the causal bound. For a query row at position p of a
 * sequence with L keys, q head h, kv head g = h / (num_q_heads / num_kv_heads):
 *   z_j = scale * q . k_j
 *   z_j = softcap * tanh(z_j / softcap)              when softcap > 0
 *   z_j = z_j - alibi_slopes[h] * |p - j|            when alibi_slopes is given
 *   key j is visible when  j < L,  j >= key_start,  and
 *       ( j < prefix_len  or  ( j <= p  and  (window == 0 or j > p - window) ) )
 *   or, with prefix_causal = 1,  when  j < L,  j >= key_start,  j <= p,  and
 *       ( j < prefix_len  or  window == 0  or  j > p - window )
 *   out = sum over visible j of softmax(z)_j v_j;  an all-zero row when no key is visible
 * softcap bounds the scores; alibi_slopes is a linear distance bias; window a sliding window that
 * counts the row's own key; prefix_len names the first keys of a sequence that every row of it
 * sees: rows before them included (prompts whose prefix is attended in both directions), or, with
 * prefix_causal, only rows at or behind them (the first tokens of a causal model that stay visible
 * under a window). The two differ for prefill rows inside the prefix only. key_start is the first
 * key a row may see (a document mask for packed documents: where the row's document starts).
 *   softcap       0 (none) or a positive finite number
 *   alibi_slopes  NULL or [num_q_heads] fp32
 *   window        0 (none) or a positive number of keys
 *   key_start     NULL or int32 per query row: [num_seqs] for decode, [total_query_tokens] for
 *                 prefill; a negative entry counts as 0, one past the row's keys leaves it empty
 *   prefix_len    NULL or [num_seqs] int32; clamped to [0, seq_lens[i]]
 *   prefix_causal 0 or 1; without prefix_len it changes nothing
 * All arrays are device arrays, 4-byte aligned. A NULL descriptor, or one of zeros, gives plain
 * causal attention.
 *
 * Pages (block-table entries) none of whose keys is visible to a row of the call may be freed:
 * their table entries must only be valid ids (the null block, as pa_bm_release_behind leaves
 * them), and their cells may hold anything. K of an invisible key never reaches a result. V of a
 * key that no row of the sequence sees never does either; V of a key that some rows of the call
 * see and others do not must be finite for the others.
 * Scores, softmax statistics and outputs are accumulated in fp32; on bf16 data the probabilities
 * are rounded to bf16 for the tensor-core product with V, and outputs are rounded once.
 */
typedef struct {
    float softcap;
    int32_t window;
    const float* alibi_slopes;
    const int32_t* key_start;
    const int32_t* prefix_len;
    int32_t prefix_causal;
} pa_score;

/*
 * pa_decode_scored: pa_decode_bs with scored attention; one query row per sequence, at position
 * seq_lens[i] - 1. Supported: bf16 or fp32, head_dim 64 or 128, any number of q heads per kv
 * head, block sizes 16, 32, 64 and 128.
 *   score      host pointer to the descriptor above (its arrays are device arrays), or NULL
 *   workspace  >= pa_decode_scored_workspace_size(...) bytes, 16-byte aligned, zero-filled before
 *              its first use; every call that completes without a device error leaves it ready
 *              for the next one. Calls that use the same workspace must not overlap on the GPU.
 * The workspace size does not depend on the block size or on the descriptor.
 * No counterpart exists on the source pages; the calls stand beside pa_decode_bs and
 * pa_prefill_chunk_bs for models whose attention has such scores.
 */
PA_API size_t pa_decode_scored_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                              int32_t head_dim, int32_t max_seq_len, pa_dtype dtype);
PA_API pa_status pa_decode_scored(void* out, const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                  int32_t num_seqs, int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads,
                                  int32_t head_dim, int32_t num_blocks, int32_t block_size, float scale,
                                  const pa_score* score, pa_dtype dtype, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * pa_prefill_scored: pa_prefill_chunk_bs with scored attention; chunk row r of sequence i sits at
 * position seq_lens[i] - C_i + r. A chunk longer than max_chunk_len or than its sequence sets
 * PA_DEVERR_LEN_RANGE and leaves its rows unwritten. workspace: as for pa_decode_scored, sized by
 * pa_prefill_scored_workspace_size (may be NULL when that is 0, which it is for short contexts); a
 * size found for some num_seqs and max_chunk_len serves every call with the same heads, head_dim and
 * dtype up to its max_seq_len. Calls with few rows on long contexts split their keys among the SMs and
 * join the parts there. Supported: as pa_decode_scored.
 */
PA_API size_t pa_prefill_scored_workspace_size(int32_t num_seqs, int32_t max_chunk_len, int32_t num_q_heads,
                                               int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len,
                                               pa_dtype dtype);
PA_API pa_status pa_prefill_scored(void* out, const void* q, const void* k_cache, const void* v_cache,
                                   const int32_t* block_table, int32_t max_blocks_per_seq, const int32_t* seq_lens,
                                   const int32_t* query_start_loc, int32_t num_seqs, int32_t max_chunk_len,
                                   int32_t max_seq_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                   int32_t num_blocks, int32_t block_size, float scale, const pa_score* score,
                                   pa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * 4-bit pools: K and V held in 4 bits and a shared scale, 9/32 of the bytes of bf16. A value is
 *   code * scale * factor
 * with the code in e2m1 (+-{0, 0.5, 1, 1.5, 2, 3, 4, 6}: bit 3 the sign, bits 0-2 the magnitude's
 * index), the scale in e4m3, shared by 16 consecutive dims of a token's head row, and the pool's
 * factor k_scale or v_scale: a power of two between 2^-24 and 2^24 that the caller keeps with the
 * pool and passes to every call (1 serves values whose groups have a largest magnitude between
 * 0.01 and 2688).
 *   k_cache, v_cache   [num_blocks][num_kv_heads][BS / 16] pages of 9 * head_dim bytes, 16-byte
 *                      aligned: 16 tokens' rows of head_dim / 2 bytes of codes (dim 2 i in the low
 *                      half of byte i), then 16 tokens' rows of head_dim / 16 scales
 *   storing x          y = x / factor;  scale = e4m3(max over the group |y| / 6), nearest, ties to
 *                      even, at most 448;  code = e2m1(y / scale), nearest, ties to even, magnitude
 *                      at most 6;  all codes 0 when the scale is 0. Infinities saturate; a NaN takes
 *                      no part in the maximum and is stored as some number.
 * Such pools take pa_rotate_and_cache, pa_decode_fp4, pa_prefill_fp4 and pa_gather_fp4; pa_move_blocks
 * (whole blocks) and pa_bm_num_blocks_for_memory with dtype PA_FP4; and every block-manager call.
 * head_dim 64 or 128. No counterpart on the source pages.
 */

/*
 * pa_rotate_and_cache: new tokens on their way into the pool. For token t at position
 * p = positions[t], with c_i = cos_sin[p][i] and s_i = cos_sin[p][rotary_dim / 2 + i]:
 *   interleaved 0   (x_i, x_(i + rotary_dim/2)) -> (x_i c_i - x_(i + rotary_dim/2) s_i,
 *                                                   x_(i + rotary_dim/2) c_i + x_i s_i)
 *   interleaved 1   (x_2i, x_(2i+1))            -> the same with these two
 * for i < rotary_dim / 2; dims from rotary_dim on stay. Every head of q[t] rotated goes to q_out[t];
 * every kv head of k[t] rotated and of v[t] goes to slot slot_mapping[t] of the pools, as
 * pa_reshape_and_cache writes them (a negative slot: q_out only).
 * The rotation is computed in fp32 and rounded once to dtype. Into a 4-bit pool k is first rounded to
 * fp32 (from a sum of about 45 bits) and to dtype, then stored: the bytes are those of storing the
 * exactly rotated k so rounded (one rotated in fp32 may lie on the other side of a border of dtype).
 *   q_out, q      [num_tokens] rows of [num_q_heads][head_dim], q_out_stride and q_stride elements
 *                 apart; q_out may be q itself (same stride). Both NULL with num_q_heads 0.
 *   k, v          [num_tokens] rows of [num_kv_heads][head_dim], k_stride and v_stride apart
 *                 (views of a packed projection, for example). Rows must be 16-byte aligned: strides
 *                 are multiples of 16 bytes and at least a row (one token: any stride).
 *   positions     [num_tokens] int64 in [0, num_positions); another one sets PA_DEVERR_POSITION, and
 *                 the token is left out (q_out row and slot keep what they held)
 *   cos_sin       [num_positions][rotary_dim] fp32
 *   rotary_dim    a multiple of 16 up to head_dim (another positive value: PA_ERR_UNSUPPORTED)
 *   slot_mapping  [num_tokens] int64, under pa_reshape_and_cache's rules
 *   cache_dtype   dtype, or PA_FP4; k_scale and v_scale are read for PA_FP4 only
 * Supported: bf16 or fp32, head_dim 64 or 128, block sizes 16, 32, 64 and 128. int64 arrays are 8-byte
 * aligned.
 */
typedef struct {
    void* q_out;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_out_stride, q_stride, k_stride, v_stride;
    const int64_t* positions;
    const float* cos_sin;
    int32_t num_positions, rotary_dim, interleaved;
    void* k_cache;
    void* v_cache;
    const int64_t* slot_mapping;
    int32_t num_tokens, num_q_heads, num_kv_heads, head_dim, num_blocks, block_size;
    pa_dtype dtype, cache_dtype;
    float k_scale, v_scale;
} pa_rotate;

PA_API pa_status pa_rotate_and_cache(const pa_rotate* rotate, void* stream);

/*
 * A call of pa_decode_fp4 or pa_prefill_fp4. Fields as the arguments of pa_decode_bs and
 * pa_prefill_chunk_bs; k_cache and v_cache are 4-bit pools with their factors, dtype (bf16 or fp32) is
 * that of q and out. query_start_loc and max_chunk_len are read by pa_prefill_fp4 only.
 */
typedef struct {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* query_start_loc;
    void* workspace;
    size_t workspace_bytes;
    int32_t max_blocks_per_seq, num_seqs, max_chunk_len, max_seq_len;
    int32_t num_q_heads, num_kv_heads, head_dim, num_blocks, block_size;
    pa_dtype dtype;
    float scale, k_scale, v_scale;
} pa_fp4_attention;

/*
 * pa_decode_fp4: pa_decode_bs over 4-bit pools: K_i[j] and V_i[j] are the values described above. Any
 * number of q heads per kv head. Products run on the tensor cores in fp16 (on the CUDA cores in fp32 where
 * num_kv_heads * ceil(heads per kv head / 16) exceeds 16384, or that times max_seq_len / 16 nears 2^31;
 * pa_prefill_fp4: above 128 q heads per kv head or 65535 sequences), which holds the pool's values
 * exactly; sums and softmax statistics are fp32. bf16 queries: each q head's row is scaled by a power of
 * two to fp16, weights are rounded to fp16 (11 bits). fp32 queries: both are sums of two fp16 numbers, 22 bits.
 * What is 2^-39 below a row's largest magnitude, or 2^-32 below the weights' sum, is lost.
 * workspace: >= pa_decode_fp4_workspace_size(...) bytes, under the rules of pa_decode_scored's.
 */
PA_API size_t pa_decode_fp4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t max_seq_len, pa_dtype dtype);
PA_API pa_status pa_decode_fp4(const pa_fp4_attention* call, void* stream);

/*
 * pa_prefill_fp4: pa_prefill_chunk_bs over 4-bit pools, with pa_decode_fp4's values and arithmetic. A
 * chunk longer than max_chunk_len or than its sequence sets PA_DEVERR_LEN_RANGE and leaves its rows
 * unwritten. workspace: >= pa_prefill_fp4_workspace_size(...) bytes, under the rules of
 * pa_prefill_scored's (may be NULL when that is 0).
 */
PA_API size_t pa_prefill_fp4_workspace_size(int32_t num_seqs, int32_t max_chunk_len, int32_t num_q_heads,
                                            int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len,
                                            pa_dtype dtype);
PA_API pa_status pa_prefill_fp4(const pa_fp4_attention* call, void* stream);

/*
 * pa_gather_fp4: rows of 4-bit pools as values, e.g. to move a sequence into another pool:
 * k_out[i] and v_out[i] ([num_slots][num_kv_heads][head_dim], dtype bf16 or fp32, which hold the
 * values exactly) are what slot slots[i] (int64) holds. A negative slot gives a row of zeros; one
 * outside the pool too, and sets PA_DEVERR_SLOT_RANGE. Slots may repeat.
 */
typedef struct {
    void* k_out;
    void* v_out;
    const void* k_cache;
    const void* v_cache;
    const int64_t* slots;
    int32_t num_slots, num_kv_heads, head_dim, num_blocks, block_size;
    pa_dtype dtype;
    float k_scale, v_scale;
} pa_fp4_rows;

PA_API pa_status pa_gather_fp4(const pa_fp4_rows* rows, void* stream);

/*
 * pa_get_device_errors: read the device error word of the current device (PA_DEVERR_*
 * bits OR-ed by the kernels since the last clear) into *errors, and clear it when
 * `clear` is non-zero. Synchronises the current device. The library owns the word.
 */
PA_API pa_status pa_get_device_errors(uint32_t* errors, int32_t clear);

/*
 * pa_debug_set_wait_drill: a test hook for the kernels' bounded waits; the source pages have
 * no counterpart. Every pipeline wait in the tensor-core kernels gives up after a time limit
 * (1 s), raises PA_DEVERR_WAIT_TIMEOUT, lets the copies it already issued land, frees its
 * tensor memory and returns without writing its results. The drill makes one such wait run
 * out on purpose, with nothing in flight that the kernel abandons:
 *   PA_DRILL_OFF              normal operation (limit back to 1 s; limit_ns is ignored)
 *   PA_DRILL_DECODE_STAGE     bf16 grouped decode (pa_decode, pa_decode_append, pa_step):
 *                             the warp that holds the first page of the work list announces
 *                             16 bytes more on its first ring stage than its copies bring;
 *                             pa_decode_fp4: likewise, on its first step of K
 *   PA_DRILL_PREFILL_K_TILE   tensor-core prefill (pa_prefill_chunk, pa_step): the CTA of the
 *                             first Q-tile pair of kv head 0 of the longest sequence announces
 *                             16 bytes more on its first K tile; pa_prefill_fp4 on the tensor cores: the
 *                             CTA of kv head 0 that is first in the order of work (up to 256 entries: the
 *                             longest; else the first sequence's) likewise
 * While a drill is on, limit_ns (1000 .. 10^9) is the wait limit of those kernels. The setting
 * is process-wide and is read when a kernel is launched (a captured graph keeps the values of
 * its capture). After a drilled call the results of that call are invalid and its
 * workspace must be zero-filled again before its next use. Returns PA_ERR_INVALID_ARG for an
 * unknown kind or a limit out of range, else PA_OK.
 */
#define PA_DRILL_OFF 0
#define PA_DRILL_DECODE_STAGE 1
#define PA_DRILL_PREFILL_K_TILE 2
PA_API pa_status pa_debug_set_wait_drill(int32_t kind, uint64_t limit_ns);

/*
 * pa_debug_decode_slices: a test hook with no counterpart in the source pages; host only, no
 * device call. The bf16 grouped decode kernel cuts its work list of `units` (sequence, kv head,
 * 16-token page) units into `ctas` contiguous slices, one per CTA, and its last `light_ctas`
 * CTAs (the ones that start last when launches overlap) get `light_units` units fewer than the
 * others, when every slice still gets a unit; otherwise the slices are equal. This writes the
 * first unit of each slice to starts[0..ctas] (starts[ctas] = units) and, if `owners` is not
 * null, the slice that holds unit u to owners[u] for u < units, computed by the same code as
 * the kernel's. Errors: PA_ERR_INVALID_ARG for units outside [0, 2^31), ctas < 1 or a null
 * `starts`. Both arrays belong to the caller.
 */
PA_API pa_status pa_debug_decode_slices(int64_t units, int32_t ctas, int32_t light_ctas, int32_t light_units,
                                        int64_t* starts, int32_t* owners);

/* pa_status_string: static, human-readable name of a status code. */
PA_API const char* pa_status_string(pa_status status);

/*
 * ==========================================================================================
 * Block manager (host side): which physical blocks each request owns
 * ==========================================================================================
 * Host memory only, no device calls; one manager per KV pool; not thread-safe (one caller at
 * a time). It produces the block-table rows and slot mappings the kernels above read.
 *
 * Model ("vLLM: what PagedAttention turned into", "The block pool, and the two tricks in it"
 * and "What a block hash actually is"; "vLLM Internals", section 1.2):
 *   - Block 0 is taken at construction as the null block and never handed out.
 *   - Free blocks sit in one eviction-ordered queue; new blocks come from its front. A freed
 *     block without a hash goes to the front (reused first), one with a hash to the back
 *     (evicted last). A request's blocks are freed tail first.
 *   - A freed block keeps its hash and can still be hit; it leaves the cache only when it is
 *     taken for new content.
 *   - Block hash: SHA-256(parent hash || the block's 16 token ids as int32 little-endian ||
 *     extra key), chained from SHA-256(hash_seed); the extra key is the request's salt, on
 *     the first block only; the cache key is hash || group id 0 (4 bytes, big-endian).
 *   - A new request reuses the longest run of cached full blocks of its prompt (stopping at
 *     the first miss), at most (n_tokens - 1) / 16 of them, so at least one token is left to
 *     compute.
 *   - Blocks are reference counted. pa_bm_fork makes a request that shares every block of its
 *     parent (parallel sampling stores the prompt once); appending into a shared, partly
 *     filled last block first moves the request to a private copy, whose (source,
 *     destination) pair waits in the manager until pa_bm_take_copies hands it to
 *     pa_copy_blocks, which must run before the request's next K/V write.
 *   - A full block is entered into the cache once pa_bm_commit reports its K/V computed.
 * Calls that fail return a status and change nothing.
 */
typedef struct pa_block_manager pa_block_manager;

/* A manager for a pool of num_blocks (>= 2) blocks; enable_caching 0 disables prefix reuse;
 * hash_seed NULL = "paged-kv-none-hash". Free with pa_bm_destroy. */
PA_API pa_status pa_bm_create(int32_t num_blocks, int32_t enable_caching, const char* hash_seed,
                              pa_block_manager** out);
/* The same for blocks of block_size tokens (16, 32, 64 or 128; another positive size returns
 * PA_ERR_UNSUPPORTED): every "16" in the descriptions below reads block_size (hash input,
 * prefix-hit cap, slots). */
PA_API pa_status pa_bm_create_bs(int32_t num_blocks, int32_t block_size, int32_t enable_caching,
                                 const char* hash_seed, pa_block_manager** out);
PA_API void pa_bm_destroy(pa_block_manager* bm);
/* Blocks in the free queue (cached-but-free blocks included); -1 for a NULL manager. */
PA_API int32_t pa_bm_num_free_blocks(const pa_block_manager* bm);

/* A new request with its prompt tokens (host int32[n_tokens], n_tokens >= 1) and optional
 * salt bytes; allocates ceil(n_tokens / 16) blocks, the cached prefix ones shared;
 * *num_cached_tokens = tokens whose K/V is already in the pool (a multiple of 16).
 * PA_ERR_INVALID_ARG for a known req_id; PA_ERR_NO_SPACE when the pool is short. */
PA_API pa_status pa_bm_add_request(pa_block_manager* bm, int64_t req_id, const int32_t* tokens, int32_t n_tokens,
                                   const uint8_t* salt, int32_t salt_len, int32_t* num_cached_tokens);
/* Appends n tokens (e.g. one per decode step), allocating blocks at block boundaries and
 * copying a shared, partly filled last block first (copy-on-write). */
PA_API pa_status pa_bm_append_tokens(pa_block_manager* bm, int64_t req_id, const int32_t* tokens, int32_t n);
/* The first num_computed_tokens tokens of the request have their K/V in the pool: its full
 * blocks among them are hashed and entered into the prefix cache. */
PA_API pa_status pa_bm_commit(pa_block_manager* bm, int64_t req_id, int32_t num_computed_tokens);
/* child_id shares every block (and the tokens) of parent_id. */
PA_API pa_status pa_bm_fork(pa_block_manager* bm, int64_t parent_id, int64_t child_id);
/* Releases the request's blocks, tail first. */
PA_API pa_status pa_bm_free_request(pa_block_manager* bm, int64_t req_id);

/* The request's block-table row: block_ids[i] for i < capacity, padded with the null block;
 * *num_blocks = blocks the request holds (PA_ERR_NO_SPACE if more than capacity). */
PA_API pa_status pa_bm_get_blocks(const pa_block_manager* bm, int64_t req_id, int32_t* block_ids, int32_t capacity,
                                  int32_t* num_blocks);
/* Slots (block * 16 + offset) of positions first_pos .. first_pos + n - 1 of the request,
 * which must lie inside its blocks. */
PA_API pa_status pa_bm_slot_mapping(const pa_block_manager* bm, int64_t req_id, int32_t first_pos, int32_t n,
                                    int64_t* slots);
/* Moves up to capacity pending copy-on-write pairs (oldest first) into src / dst;
 * PA_ERR_NO_SPACE if some remain. */
PA_API pa_status pa_bm_take_copies(pa_block_manager* bm, int32_t* src, int32_t* dst, int32_t capacity,
                                   int32_t* n_copies);
/* Gives back the request's blocks that lie wholly in positions [keep, first_pos) (a sliding window
 * has passed them; the first `keep` tokens stay): their entries become the null block, the blocks
 * are released tail first as by pa_bm_free_request (a hashed one can still be hit by another
 * request). *num_released = blocks given back by this call. first_pos at most the request's token
 * count, keep >= 0. Positions given back have no slots: pa_bm_slot_mapping refuses them. */
PA_API pa_status pa_bm_release_behind(pa_block_manager* bm, int64_t req_id, int32_t first_pos, int32_t keep,
                                      int32_t* num_released);
/* Changes the pool's size to num_blocks (>= 2). Growing adds free blocks at the back of the queue.
 * Shrinking moves every held block with id >= num_blocks to a free block below it (taken in queue
 * order; a cached one is evicted), in all requests' lists and with its hash, and removes the blocks
 * from num_blocks on. The moves come out as (src[i], dst[i]), i < *n_moves, both strictly
 * ascending and every dst below every src; the caller hands them to pa_move_blocks before the next
 * access to the pool. PA_ERR_NO_SPACE when fewer free blocks are left below than moves are needed,
 * or `capacity` is below *n_moves (set to the moves needed); PA_ERR_INVALID_ARG while
 * copy-on-write pairs wait for pa_bm_take_copies. A failed call changes nothing. */
PA_API pa_status pa_bm_resize(pa_block_manager* bm, int32_t num_blocks, int32_t* src, int32_t* dst, int32_t capacity,
                              int32_t* n_moves);
/* Inspection: the free queue from front to back, and one block's reference count and hash. */
PA_API pa_status pa_bm_free_queue(const pa_block_manager* bm, int32_t* order, int32_t capacity, int32_t* n);
PA_API pa_status pa_bm_block_info(const pa_block_manager* bm, int32_t block_id, int32_t* ref_count,
                                  uint8_t* hash32, int32_t* has_hash);
/* Pool size for a memory budget: floor(utilization * free_bytes / per-block bytes over all
 * layers, K and V) ("vLLM: what PagedAttention turned into", "Checking the 96.3%": the pool
 * is sized once from a utilisation fraction of free memory); -1 on a bad argument. */
PA_API int64_t pa_bm_num_blocks_for_memory(size_t free_bytes, double utilization, int32_t num_layers,
                                           int32_t num_kv_heads, int32_t head_dim, pa_dtype dtype);
/* The same for blocks of block_size tokens (16, 32, 64 or 128; -1 otherwise). dtype of both: PA_FP4 for 4-bit
 * pools (head_dim then a multiple of 64). */
PA_API int64_t pa_bm_num_blocks_for_memory_bs(size_t free_bytes, double utilization, int32_t num_layers,
                                              int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                              pa_dtype dtype);
/* SHA-256 (FIPS 180-4) of n bytes, as the block hashes use it. */
PA_API pa_status pa_sha256(const uint8_t* data, size_t n, uint8_t* out32);

/*
 * pa_copy_blocks: for each of the n_pairs (src, dst) block-id pairs in block_pairs (device
 * int32 [n_pairs][2]), copy block src of k_cache and of v_cache, every kv head, into block
 * dst (the copy-on-write pairs of the block manager). Pairs must not chain (no dst is another
 * pair's src); src == dst is skipped. Out-of-range ids are not copied and set
 * PA_DEVERR_BLOCK_RANGE. Asynchronous on `stream`.
 */
PA_API pa_status pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* block_pairs, int32_t n_pairs,
                                int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, pa_dtype dtype,
                                void* stream);

/* pa_copy_blocks with block_size (see the block-size variants above). */
PA_API pa_status pa_copy_blocks_bs(void* k_cache, void* v_cache, const int32_t* block_pairs, int32_t n_pairs,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size,
                                   pa_dtype dtype, void* stream);

/*
 * pa_move_blocks: copy pages between physical blocks in every layer's pools at once, and rewrite
 * block tables to follow. For each (src, dst) pair of block_pairs (device int32 [n_pairs][2]) and
 * every pool: block src, every kv head, is copied into block dst. Forked requests' last pages
 * (copy-on-write), compaction after pa_bm_resize, and reordering of pages are such copies; a
 * model has two pools per layer, and one launch serves all of them.
 *   pools        host array of num_pools device pointers, each [num_blocks][num_kv_heads]
 *                [block_size][head_dim], 16-byte aligned (K and V pools alike); the array is read
 *                during the call only
 *   dtype        the pools' type; PA_FP4 for 4-bit pools, whose blocks move whole (`tokens` NULL, else
 *                PA_ERR_UNSUPPORTED)
 *   tokens       NULL (whole blocks) or device int32 [n_pairs]: only the first tokens[i] tokens of
 *                each head's page are copied (the filled part of a partly filled block); clamped
 *                to [0, block_size]
 *   block_table  NULL or device int32 [num_seqs][max_blocks_per_seq]: every entry equal to some
 *                pair's src becomes that pair's dst, among the first ceil(seq_lens[i] / block_size)
 *                entries of row i (clamped to the row); other entries keep their value. The
 *                pairs' src must then be strictly ascending (as pa_bm_resize returns them); pairs
 *                that are not set PA_DEVERR_PAIR_ORDER, and the table is then unspecified.
 *   seq_lens     device int32 [num_seqs], needed with block_table
 * Several pairs may share a src. Every dst must be distinct, and no dst may be another pair's src
 * or a block that a kernel running at the same time reads. src == dst is skipped; ids outside
 * [0, num_blocks) are not copied and set PA_DEVERR_BLOCK_RANGE. Asynchronous on `stream`.
 * No counterpart on the source pages beyond the copy-on-write of pa_copy_blocks.
 */
PA_API pa_status pa_move_blocks(void* const* pools, int32_t num_pools, int32_t num_kv_heads, int32_t head_dim,
                                int32_t num_blocks, int32_t block_size, pa_dtype dtype, const int32_t* block_pairs,
                                int32_t n_pairs, const int32_t* tokens, int32_t* block_table,
                                int32_t max_blocks_per_seq, const int32_t* seq_lens, int32_t num_seqs, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PA_H */
