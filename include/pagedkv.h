/*
 * pagedkv.h -- C ABI of libpagedkv.so, the GB300 (sm_103a) hot path of a
 * paged KV cache: slot mapping, the cache write, and paged attention over a
 * block-table-indexed pool for one mixed continuous-batching step.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Pointers named as device buffers are CUDA device pointers on the current
 *   device, owned by the caller. The library never allocates, frees or keeps
 *   them past the call, and never synchronises the stream inside a compute
 *   call: work is only enqueued on `stream` (a cudaStream_t passed as void*;
 *   NULL = the legacy default stream).
 * - bf16 tensors are IEEE bfloat16 bit patterns. Row strides are counted in
 *   elements and must keep every row 16-byte aligned.
 * - Every call returns PKV_OK (0) or a negative PKV_ERR_* status. Argument
 *   checks run on the host before anything is enqueued; a failed check
 *   enqueues nothing. A CUDA launch error returns PKV_ERR_CUDA and
 *   pkv_last_cuda_error() gives its text.
 * - Bad *contents* of device arrays (a slot or block id outside the pool,
 *   inconsistent lengths) cannot be seen by the host without a sync. Kernels
 *   skip such entries instead of touching memory out of range and set bits in
 *   a sticky per-device error word, read by pkv_get_device_errors().
 *
 * Pool layout (the pages' physical KV cache, "vllm v1 源码精读（三）", §3.3):
 *   kv_cache[num_blocks][2][block_size][num_kv_heads][head_dim], bf16,
 *   contiguous; index 0 of the second dimension holds K, 1 holds V.
 *   block_size (B) is 8, 16 or 32 tokens: 16 is the pages' default and 8
 *   and 32 the two other points of "vLLM 架构源码解析（一）" §5.1 (less
 *   last-block waste vs fewer block-table entries); other sizes return
 *   PKV_ERR_UNSUPPORTED. num_blocks * 2 * B must stay below 2^31.
 *   head_dim must be 64 or 128.
 *
 * Launches: every kernel is launched with programmatic stream serialization.
 * A kernel may start (set up barriers, allocate tensor memory, fetch the
 * descriptors passed as its own parameters) while the previous kernel in the
 * stream is still running, and it waits for that kernel to complete -- and
 * its writes to be visible -- before reading any buffer. Work the caller
 * queued earlier on the stream is therefore seen as with plain stream order.
 * The write calls (pkv_slot_mapping, pkv_paged_kv_write,
 * pkv_slot_mapping_and_write), the attention calls that take the caller's
 * workspace (pkv_paged_attention, pkv_paged_attention_with_write), the table
 * calls (pkv_build_step_tables, pkv_release_blocks) and every pkv_quant_ call that
 * takes a stream can be recorded into a CUDA graph.
 */
#ifndef PAGEDKV_H_
#define PAGEDKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_ABI_VERSION 2

/* status codes */
#define PKV_OK 0
#define PKV_ERR_NULL_POINTER (-1) /* a required pointer is NULL             */
#define PKV_ERR_BAD_SHAPE (-2)    /* a size or count is out of range         */
#define PKV_ERR_UNSUPPORTED (-3)  /* valid but not built (block size, d, G)  */
#define PKV_ERR_MISALIGNED (-4)   /* pointer or stride not 16-byte aligned   */
#define PKV_ERR_WORKSPACE (-5)    /* workspace missing or too small          */
#define PKV_ERR_CUDA (-6)         /* a CUDA runtime / driver call failed     */
#define PKV_ERR_DEVICE (-7)       /* the current device is not sm_103        */
#define PKV_ERR_SCRATCH_LIMIT (-8) /* the call needs more scratch than the
                                      library's built-in array holds (see
                                      pkv_paged_attention_static_workspace)    */

/* bits of the sticky device error word */
#define PKV_DEVERR_SLOT_RANGE 0x1u  /* slot >= num_blocks * block_size: row skipped */
#define PKV_DEVERR_BLOCK_RANGE 0x2u /* table entry outside [0, num_blocks) in the
                                       used range: its keys are masked out       */
#define PKV_DEVERR_LENGTHS 0x4u     /* query_start_loc / seq_lens /
                                       num_computed_tokens inconsistent, or a
                                       sequence needs more than
                                       max_blocks_per_req blocks                 */
#define PKV_DEVERR_TIMEOUT 0x8u     /* an on-chip wait (TMA / tensor core) gave
                                       up after its time limit                    */
#define PKV_DEVERR_SHARED 0x10u     /* the shared-prefix hint of
                                       pkv_attention_options did not hold for
                                       some request; it was attended without
                                       the hint (results unaffected)            */
#define PKV_DEVERR_NO_BLOCKS 0x20u  /* pkv_build_step_tables: the free queue
                                       held too few blocks for some request      */
#define PKV_DEVERR_REF_COUNT 0x40u  /* pkv_release_blocks: a block was released
                                       more often than it was held               */
#define PKV_DEVERR_CHUNK_KEYS 0x80u /* 8-bit pool: the workspace holds too few
                                       chunk keys for the step; keys were masked
                                       out                                       */

/* Shape of the physical pool. */
typedef struct pkv_cache_layout {
  int32_t num_blocks;   /* physical blocks in the pool, >= 1                  */
  int32_t block_size;   /* tokens per block: 8, 16 or 32                       */
  int32_t num_kv_heads; /* kv heads per token                                 */
  int32_t head_dim;     /* 64 or 128                                          */
} pkv_cache_layout;

/* Scores and masks other than plain causal attention. For the query row t of
 * request r at position p = num_computed_tokens[r] + i (t = query_start_loc[r]
 * + i) and q head h, with x_j = scale * q . k_j:
 *   score_j = cap(x_j) - alibi_slopes[h] * |p - j|,
 *   cap(x)  = softcap * tanh(x / softcap), or x when softcap is 0,
 * and the softmax runs over the keys key_begin[t] <= j < key_end[t]. A row
 * whose range holds no key gets zeros. The ranges state, among others,
 *   - documents packed into one sequence: key_begin = the start of the
 *     document that holds p;
 *   - a prefix that is seen in both directions: key_end = max(p + 1, prefix
 *     length);
 *   - a sliding window of W tokens: key_begin = p - W + 1;
 *   - padding that sees nothing: key_end <= key_begin.
 * The cache blocks in front of a row's (or a tile of rows') first key and
 * behind its last one are not read: their table entries may be stale or -1.
 * Masked keys never reach the output, whatever their K and V rows hold.
 * With a softcap up to 51 and no slopes, requests of several new tokens are
 * summed without a maximum taken off the scores: where all scores of a row lie
 * at the cap, values above 2^32 in size may overflow, and those below 2^-30
 * are accurate to 2^-50 absolute only.
 * Every field is off at zero. The pages name no such scores; the entry points
 * are those of plain attention (pkv_attention_options). */
typedef struct pkv_score_options {
  float softcap;             /* 0 = off, else softcap and scale / softcap both in
                                [1e-30, 1e30] (else PKV_ERR_BAD_SHAPE)          */
  const float* alibi_slopes; /* device fp32 [num_q_heads], finite; NULL = off.
                                Sizes above 1e28 count as 1e28. The bias is an
                                fp32 number: 2^-24 of slope * distance is its
                                rounding, which matters where the farthest keys
                                weigh most (negative slopes)                    */
  const int32_t* key_begin;  /* device int32 [num_tokens]; NULL = 0; values
                                below 0 count as 0                              */
  const int32_t* key_end;    /* device int32 [num_tokens]; NULL = p + 1; values
                                above seq_lens[r] count as seq_lens[r]. May lie
                                past p + 1: the keys of the step's later tokens
                                are in the cache by then                        */
  int32_t reserved[4];       /* must be zero                                    */
} pkv_score_options;

/* Optional tuning and tracing of pkv_paged_attention; pass NULL for the
 * defaults. */
typedef struct pkv_attention_options {
  /* Ranges the step's decode KV stream of (request, 16-key chunk) positions
   * is cut into, one CTA each (split-KV). 0 = one full wave of the device,
   * or fewer when the hints bound the stream below that (num_reqs *
   * ceil(max_seq_len / 16)). A single range means no split at all; tests use
   * other values to vary the partitioning. */
  int32_t decode_splits;
  /* Shared prefix of a run of decode requests (prefix caching: "vLLM
   * 架构源码解析（一）" §4.3.1, blocks with ref_cnt > 1 at the head of
   * several block tables). shared_num_reqs > 0 declares that the requests
   * shared_first_req .. shared_first_req + shared_num_reqs - 1 are decodes
   * (one new token each) whose first shared_prefix_len tokens live in the
   * same physical blocks: block_table[r][j] == block_table[shared_first_req][j]
   * for j < shared_prefix_len / B. The call then attends those requests'
   * query rows over the shared prefix once, as one dense tensor-core
   * contraction (rows = requests x q heads, the prefix's keys read once
   * per kv head), and each request's decode covers only its own keys past
   * the prefix, starting from that partial result. The output is the same
   * attention (shared blocks behave as private copies); only the traffic
   * changes.
   *   - shared_prefix_len: tokens, a multiple of 16 and of B, >= 16; 0 =
   *     off (then the other two fields must be 0).
   *   - The hint is checked on the device: a request of the run whose
   *     table does not start with the shared entries, or whose seq_len is
   *     not above shared_prefix_len, is attended without it; if a request of
   *     the run has a query_len other than 1 the whole run is. Either sets
   *     PKV_DEVERR_SHARED. The results stay correct in every case.
   *   - The workspace grows with shared_num_reqs
   *     (pkv_attention_workspace_size takes the same options). */
  int32_t shared_prefix_len;
  int32_t shared_first_req;
  int32_t shared_num_reqs;
  /* [0]: 0, or PKV_OPTIONS_SCORES when the struct has the field `scores` below
   * (a caller built before that field existed leaves it 0, and the library
   * then does not read past trace_events). [1]: 0, or for the calls on the 8-bit
   * pool PKV_OPTIONS_FEW_ROWS' value (see pkv_quant_few_rows). [2], [3], and [1]
   * of the other calls, must be zero. */
  int32_t reserved[4];
  /* Tracing: NULL, or PKV_TRACE_EVENTS cudaEvent_t handles (as void*) owned
   * by the caller. The call records them on `stream` around its kernels:
   * [0] before the plan kernel, [1] before the prefill kernel, [2] before
   * the decode kernel, [3] before the combine kernel, [4] after it.
   * Consecutive pairs bracket one kernel each (an empty bracket when a
   * kernel is not needed). The events keep the kernels from overlapping
   * (see "Launches" above), so a traced call can be a little slower. */
  void** trace_events;
  /* Capped, biased or range-masked scores; NULL = plain causal attention. Read
   * only when reserved[0] is PKV_OPTIONS_SCORES. A shared-prefix hint may be
   * given with it: the prefix is then attended once under each row's own
   * scores and range. */
  const pkv_score_options* scores;
} pkv_attention_options;

#define PKV_OPTIONS_SCORES 1
/* Place in reserved[] of the most new tokens of a request that a call on the 8-bit
 * pool takes on the decode kernels. */
#define PKV_OPTIONS_FEW_ROWS 1

#define PKV_TRACE_EVENTS 5

/* Library version (PKV_ABI_VERSION). */
int32_t pkv_abi_version(void);

/* Text for a status code; never NULL. */
const char* pkv_status_string(int32_t status);

/* Text of the last CUDA error this thread saw inside the library. */
const char* pkv_last_cuda_error(void);

/*
 * pkv_slot_mapping -- physical slot of every new token of the varlen batch.
 *
 * "vllm v1 源码精读（三）" §3.4: request r's i-th new token sits at position
 * pos = num_computed_tokens[r] + i and goes to
 *   slot = block_table[r][pos / block_size] * block_size + pos % block_size
 * (the page's worked examples: request 0 pos 17 -> 193, request 2 pos 32 ->
 * 144 with tables [[5,12,-1],[3,-1,-1],[7,21,9]]).
 *
 * slot_mapping        out, device int64 [num_tokens]. Token t belongs to the
 *                     request r with query_start_loc[r] <= t <
 *                     query_start_loc[r+1]; tokens at or past
 *                     query_start_loc[num_reqs] get -1 (padding). A token
 *                     whose table entry is missing or outside the pool gets
 *                     -1 and sets PKV_DEVERR_BLOCK_RANGE / _LENGTHS. Every
 *                     row of a request with inconsistent lengths
 *                     (query_start_loc[r] < 0, query_start_loc[r+1] <
 *                     query_start_loc[r] or > num_tokens,
 *                     num_computed_tokens[r] < 0, or query_start_loc[0] !=
 *                     0) gets -1 and sets PKV_DEVERR_LENGTHS; so does every
 *                     row before query_start_loc[0] when that is not 0. No
 *                     row keeps what the buffer held before the call.
 * block_table         device int32 [num_reqs][max_blocks_per_req], -1 = unused.
 * query_start_loc     device int32 [num_reqs + 1], non-decreasing, [0] = 0.
 * num_computed_tokens device int32 [num_reqs].
 * num_blocks          pool size, for the range check.
 * block_size          tokens per block: 8, 16 or 32 (else PKV_ERR_UNSUPPORTED).
 */
int32_t pkv_slot_mapping(int64_t* slot_mapping, const int32_t* block_table,
                         int32_t max_blocks_per_req,
                         const int32_t* query_start_loc,
                         const int32_t* num_computed_tokens, int32_t num_reqs,
                         int32_t num_tokens, int32_t num_blocks,
                         int32_t block_size, void* stream);

/*
 * pkv_paged_kv_write -- reshape_and_cache: store each new token's K and V rows
 * into the pool at its slot ("vLLM 架构源码解析（一）" §3.3.3 step 2;
 * "vllm v1 源码精读（三）" §3.4, reshape_and_cache_flash). A bit copy:
 *   kv_cache[s / B][0][s % B][:][:] = key[t],  [..][1][..] = value[t]
 * for every t with s = slot_mapping[t] >= 0 (B = layout.block_size).
 * Negative slots are skipped; slots >= num_blocks * B are skipped and set
 * PKV_DEVERR_SLOT_RANGE. Two
 * tokens with the same slot race (undefined which wins).
 *
 * kv_cache      in/out, device bf16 pool (layout above).
 * key, value    device bf16 [num_tokens][num_kv_heads][head_dim]; row t starts
 *               at key + t * key_row_stride (0 = num_kv_heads * head_dim).
 * slot_mapping  device int64 [num_tokens].
 */
int32_t pkv_paged_kv_write(void* kv_cache, const void* key, const void* value,
                           int64_t key_row_stride, int64_t value_row_stride,
                           const int64_t* slot_mapping, int32_t num_tokens,
                           pkv_cache_layout layout, void* stream);

/*
 * pkv_slot_mapping_and_write -- pkv_slot_mapping and pkv_paged_kv_write fused
 * into one kernel (the pages compute the slot mapping on the device and then
 * store the rows: "vllm v1 源码精读（三）" §3.4; "vLLM 架构源码解析（一）"
 * §3.3.3 step 2). Each new token's slot is computed as pkv_slot_mapping
 * defines it, and its K and V rows are stored there as pkv_paged_kv_write
 * does, with one launch instead of two.
 *
 * slot_mapping  out, device int64 [num_tokens], or NULL (not stored). For a
 *               non-decreasing query_start_loc it receives exactly what
 *               pkv_slot_mapping writes; a token with slot -1 is not written.
 *               Tokens are assigned to requests by searching
 *               query_start_loc, so where it decreases (inconsistent
 *               lengths, PKV_DEVERR_LENGTHS) the rows that get -1 may differ
 *               from pkv_slot_mapping's.
 * kv_cache, key, value, key_row_stride, value_row_stride, layout
 *               as pkv_paged_kv_write (layout.num_blocks is the range check).
 * block_table, max_blocks_per_req, query_start_loc, num_computed_tokens,
 * num_reqs, num_tokens   as pkv_slot_mapping.
 */
int32_t pkv_slot_mapping_and_write(void* kv_cache, const void* key, const void* value,
                                   int64_t key_row_stride, int64_t value_row_stride,
                                   int64_t* slot_mapping, const int32_t* block_table,
                                   int32_t max_blocks_per_req, const int32_t* query_start_loc,
                                   const int32_t* num_computed_tokens, int32_t num_reqs,
                                   int32_t num_tokens, pkv_cache_layout layout, void* stream);

/*
 * pkv_copy_blocks -- copy whole blocks (K and V of every kv head) between two
 * pools of the same block shape:
 *   - copy-on-write: before a new token is written into a block that other
 *     sequences also reference, the writer gets its own copy of the block
 *     ("vLLM 架构源码解析（一）" §4.3.2, parallel sampling), src_pool ==
 *     dst_pool;
 *   - swap-out / swap-in of a preempted request ("vLLM 架构源码解析（一）"
 *     §1.1, v0 preemption by swapping the KV cache to CPU memory), one pool
 *     on the device and the other in pinned host memory.
 *   dst_pool[d][...] = src_pool[s][...] for every pair (s, d): a bit copy of
 *   2 * B * num_kv_heads * head_dim bf16.
 *
 * dst_pool, src_pool  pools [num_blocks][2][B][num_kv_heads][head_dim] bf16:
 *                     device memory, or pinned host memory the device can
 *                     address with the same pointer (unified addressing).
 * dst_num_blocks, src_num_blocks  pool sizes, for the range checks.
 * block_pairs         device int32 [num_pairs][2] = (source block, destination
 *                     block). A pair out of range is skipped and sets
 *                     PKV_DEVERR_BLOCK_RANGE. Pairs with the same destination,
 *                     or a destination that is another pair's source within one
 *                     call, race (undefined contents).
 * layout              block shape; its num_blocks field is ignored.
 */
int32_t pkv_copy_blocks(void* dst_pool, int32_t dst_num_blocks, const void* src_pool,
                        int32_t src_num_blocks, const int32_t* block_pairs,
                        int32_t num_pairs, pkv_cache_layout layout, void* stream);

/*
 * pkv_attention_workspace_size -- bytes of device workspace that
 * pkv_paged_attention needs for `num_reqs` requests on the current device
 * with the given options (NULL = defaults). Returns a negative status on bad
 * arguments. The size does not depend on sequence lengths.
 */
int64_t pkv_attention_workspace_size(int32_t num_reqs, int32_t num_q_heads,
                                     pkv_cache_layout layout,
                                     const pkv_attention_options* options);

/*
 * pkv_paged_attention -- attention of one mixed step over the paged cache.
 *
 * Run it after pkv_paged_kv_write of the same step: the step's new tokens are
 * read back from the pool ("vLLM 架构源码解析（一）" §3.3.3: write, then
 * attend through the block tables; "vllm v1 源码精读（三）" §4.2: one varlen
 * call holds prefill chunks and decodes; "Inside vLLM" §3.4: each sequence
 * attends only its own tokens).
 *
 * For request r with c = num_computed_tokens[r], n = query_start_loc[r+1] -
 * query_start_loc[r] and L = seq_lens[r] = c + n: its i-th query row
 * (batch row query_start_loc[r] + i, absolute position c + i) and q head h
 * attend keys j = 0 .. c + i of kv head h / (num_q_heads / num_kv_heads):
 *   out = sum_j softmax_j(scale * q . k_j) v_j,
 * key j read from block block_table[r][j / B], offset j % B.
 * Rows with n == 1 run on the split-KV decode kernels (+ combine); rows of
 * requests with n > 1 run on the tensor-core prefill kernel.
 *
 * out            device bf16 [num_tokens][num_q_heads][head_dim], contiguous.
 *                Rows past query_start_loc[num_reqs] are not written.
 * q              device bf16 [num_tokens][num_q_heads][head_dim]; row t at
 *                q + t * q_row_stride (0 = num_q_heads * head_dim).
 * kv_cache       device bf16 pool (layout above), read only.
 * block_table    device int32 [num_reqs][max_blocks_per_req], -1 = unused;
 *                entries from ceil(L / B) on are never read;
 *                max_seq_len <= max_blocks_per_req * B.
 * seq_lens, query_start_loc, num_computed_tokens: device int32 as above.
 * num_tokens     rows of q / out (>= query_start_loc[num_reqs]).
 * max_query_len  host hint: >= every n (like max_seqlen_q).
 * max_seq_len    host hint: >= every L (like max_seqlen_k).
 * num_q_heads    multiple of num_kv_heads; num_q_heads / num_kv_heads must be
 *                1, 2, 4 or 8.
 * scale          softmax scale, positive and finite (1/sqrt(head_dim) on the
 *                pages' models); anything else is PKV_ERR_BAD_SHAPE.
 * workspace      device buffer of at least pkv_attention_workspace_size()
 *                bytes, 256-byte aligned, private to this call while it runs
 *                (no zeroing needed).
 */
int32_t pkv_paged_attention(void* out, const void* q, int64_t q_row_stride,
                            const void* kv_cache, const int32_t* block_table,
                            int32_t max_blocks_per_req, const int32_t* seq_lens,
                            const int32_t* query_start_loc,
                            const int32_t* num_computed_tokens, int32_t num_reqs,
                            int32_t num_tokens, int32_t max_query_len,
                            int32_t max_seq_len, int32_t num_q_heads, float scale,
                            pkv_cache_layout layout, void* workspace,
                            size_t workspace_bytes,
                            const pkv_attention_options* options, void* stream);

/*
 * pkv_paged_attention_with_write -- the whole step of one layer in one call:
 * the slot mapping and cache write of every new token
 * (pkv_slot_mapping_and_write) and then pkv_paged_attention over the pool
 * that now holds them, as the pages' engine does per layer ("vLLM 架构源码解析
 * （一）" §3.3.3: write the step's K/V, then attend; "Inside vLLM" §3.4-3.5:
 * one attention call over the mixed batch). The write runs in the same
 * launch as the attention's plan (its own CTAs next to the plan's), so the
 * step takes one launch fewer than the two calls.
 *
 * Arguments: those of pkv_paged_attention, plus key, value,
 * key_row_stride, value_row_stride and slot_mapping (out, may be NULL) as in
 * pkv_slot_mapping_and_write; kv_cache is written. Results, error bits and
 * the workspace are those of the two calls. A call with no attention to do
 * (num_reqs, num_tokens or max_query_len 0) still maps and writes (padding
 * rows get slot -1). With trace_events, bracket [0, 1) covers the write and
 * the plan.
 */
int32_t pkv_paged_attention_with_write(
    void* out, const void* q, int64_t q_row_stride, void* kv_cache, const void* key,
    const void* value, int64_t key_row_stride, int64_t value_row_stride, int64_t* slot_mapping,
    const int32_t* block_table, int32_t max_blocks_per_req, const int32_t* seq_lens,
    const int32_t* query_start_loc, const int32_t* num_computed_tokens, int32_t num_reqs,
    int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len, int32_t num_q_heads,
    float scale, pkv_cache_layout layout, void* workspace, size_t workspace_bytes,
    const pkv_attention_options* options, void* stream);

/*
 * pkv_paged_attention_static_workspace -- pkv_paged_attention for callers
 * that cannot allocate device memory. The pages have no counterpart to this
 * entry point; it exists for how the library is called, not for what it
 * computes.
 *
 * Some callers have no way to hand the library a workspace: a server that
 * gave all device memory to its own caching allocator and KV pool at start-up
 * and may not call cudaMalloc afterwards, a plugin inside a host framework
 * that forbids raw device allocations, or a plain C caller with no allocator
 * at all. This call takes the same arguments as pkv_paged_attention except the
 * workspace, and uses instead one scratch array compiled into the library:
 * PKV_STATIC_WORKSPACE_BYTES of device memory that every GPU which loads the
 * library holds until the process exits. It never calls cudaMalloc, cudaFree
 * or any allocating routine.
 *
 * - Size limit: if the call would need more scratch than the array holds
 *   (pkv_attention_workspace_size() > PKV_STATIC_WORKSPACE_BYTES) it returns
 *   PKV_ERR_SCRATCH_LIMIT and enqueues nothing. With the default options the
 *   Llama-3-8B layer shape (32 q / 8 kv heads, d = 128) fits about 1860
 *   requests per call on a 152-SM GB300.
 * - First call per device: it looks up the array's device address
 *   (cudaGetSymbolAddress) with that device current. The address is kept
 *   for the life of the process: do not call this entry point again on a device after
 *   cudaDeviceReset (or after its primary context was released and made
 *   anew), since the library's device memory may then sit elsewhere.
 * - Shared state: every call on a device uses the same array and leaves its
 *   contents behind. Nothing needs to start at zero (each call re-plans the
 *   whole scratch area first). Calls whose kernels overlap on the GPU (on
 *   different streams, or from different threads) race on the array and give
 *   wrong results: keep them ordered, e.g. on one stream.
 */
#define PKV_STATIC_WORKSPACE_BYTES (32u * 1024u * 1024u)

int32_t pkv_paged_attention_static_workspace(
    void* out, const void* q, int64_t q_row_stride, const void* kv_cache,
    const int32_t* block_table, int32_t max_blocks_per_req, const int32_t* seq_lens,
    const int32_t* query_start_loc, const int32_t* num_computed_tokens, int32_t num_reqs,
    int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len, int32_t num_q_heads,
    float scale, pkv_cache_layout layout, const pkv_attention_options* options,
    void* stream);

/*
 * pkv_build_step_tables -- the metadata of one step, built on the device from
 * the requests' lengths: new blocks taken from the free queue and entered in
 * the block tables, the batch's row starts, the sequence lengths and the slot
 * of every new token ("vllm v1 源码精读（三）" §3.3: allocation pops blocks
 * from the head of a free queue; §3.4: block table and slot mapping; "vLLM
 * 架构源码解析（一）" §3.3.2: positions and lengths of the batch). The outputs
 * are the arguments of pkv_paged_kv_write, pkv_paged_attention and
 * pkv_paged_attention_with_write, so a step needs no block table from the host.
 *
 * Request r with c = num_computed_tokens[r] and n = query_lens[r] holds
 * ceil(c / B) blocks and needs ceil((c + n) / B). Its new blocks are the next
 * ones of the queue, in batch order, first come, first served: if the queue
 * cannot cover what is asked for up to and including request r, then r and
 * every later request that needs a block get none. Such a request keeps its
 * rows in the batch but gets seq_lens 0, slots -1 and -1 in the entries asked
 * for, and PKV_DEVERR_NO_BLOCKS is set. The attention calls skip it (its rows
 * are not written, PKV_DEVERR_LENGTHS), and pkv_paged_kv_write skips its slots;
 * the calls that map slots themselves write those of its tokens that still fit
 * into its own last block and set PKV_DEVERR_BLOCK_RANGE for the others.
 *
 * block_table      in/out, device int32 [num_reqs][max_blocks_per_req]: the
 *                  entries [ceil(c / B), ceil((c + n) / B)) of each row are
 *                  written, no others.
 * query_start_loc  out, device int32 [num_reqs + 1].
 * seq_lens         out, device int32 [num_reqs]: c + n.
 * slot_mapping     out, device int64 [num_tokens], or NULL. Rows at or past
 *                  query_start_loc[num_reqs] get -1.
 * num_computed_tokens, query_lens   device int32 [num_reqs]. A negative length
 *                  or a sequence of more than max_blocks_per_req blocks sets
 *                  PKV_DEVERR_LENGTHS: the request keeps its rows (a negative
 *                  query length counts as 0), with seq_lens 0 and slots -1, and
 *                  takes no block. So does a batch of more than num_tokens
 *                  rows; the rows past num_tokens have no slot.
 * free_queue       device int32 [num_blocks], a ring of free block ids.
 * free_state       device int32 [2]: the ring's head and how many ids it holds.
 * free_state_out   out, device int32 [2]: the state after the step. May be
 *                  free_state itself; another buffer leaves the queue as it
 *                  was until the caller takes the new state over.
 * ref_cnt          in/out, device int32 [num_blocks], or NULL: the new blocks
 *                  get 1.
 * A state or a queue entry out of range hands out nothing (PKV_DEVERR_LENGTHS,
 * PKV_DEVERR_BLOCK_RANGE); so does -1 in the table where a request goes on in
 * a block it should have. Apart from the state, no array that is written may
 * overlap another one (PKV_ERR_BAD_SHAPE). The call can be recorded into a CUDA graph. Calls
 * that share a queue, its state, tables or counts must be ordered.
 */
int32_t pkv_build_step_tables(int32_t* block_table, int32_t max_blocks_per_req,
                              int32_t* query_start_loc, int32_t* seq_lens, int64_t* slot_mapping,
                              const int32_t* num_computed_tokens, const int32_t* query_lens,
                              int32_t num_reqs, int32_t num_tokens, const int32_t* free_queue,
                              const int32_t* free_state, int32_t* free_state_out,
                              int32_t* ref_cnt, int32_t num_blocks, int32_t block_size,
                              void* stream);

/*
 * pkv_release_blocks -- give back the blocks of requests that finished or
 * were preempted ("vLLM 架构源码解析（一）" §4.3.1: a block returns to the pool
 * when its reference count reaches zero; "vllm v1 源码精读（三）" §3.3: at the
 * tail of the free queue).
 *
 * The rows are released in the order given, each from its last block to its
 * first, so that the blocks at the head of a sequence, the ones a prefix is
 * shared by, are reused last. Every entry counts its block down by one, and a
 * block that reaches zero is appended to the queue at the place of its last
 * release. The result does not depend on the order in which the device's threads run.
 *
 * block_table      device int32 [num_reqs][max_blocks_per_req], read only: the
 *                  entries of a released row stay as they are.
 * release_rows     device int32 [num_released]: rows of the table. Several
 *                  may share blocks; a row may stand in it as often as its
 *                  blocks are held.
 * release_tokens   device int32 [num_reqs]: tokens whose blocks row r holds,
 *                  ceil(release_tokens[r] / B) entries. After
 *                  pkv_build_step_tables that is seq_lens[r], but
 *                  num_computed_tokens[r] for a request that got no blocks: its
 *                  seq_lens is 0, and to release it by that gives nothing back.
 * free_queue       in/out, free_state in, free_state_out out: as in
 *                  pkv_build_step_tables.
 * ref_cnt          in/out, device int32 [num_blocks]: how many rows hold each
 *                  block.
 * workspace        device buffer of at least pkv_release_workspace_size()
 *                  bytes, 256-byte aligned, private to this call while it
 *                  runs (no zeroing needed); may be NULL where that is 0.
 * A row or a length out of range is skipped (PKV_DEVERR_LENGTHS), as is an
 * entry out of the pool (PKV_DEVERR_BLOCK_RANGE). A block that is released more
 * often than it is held goes back once (PKV_DEVERR_REF_COUNT). Arrays must not
 * overlap, as in pkv_build_step_tables. num_released *
 * max_blocks_per_req must stay below 2^29. The call can be recorded into a
 * CUDA graph.
 */
int32_t pkv_release_blocks(const int32_t* block_table, int32_t max_blocks_per_req,
                           int32_t num_reqs, const int32_t* release_rows,
                           const int32_t* release_tokens, int32_t num_released,
                           int32_t* free_queue, const int32_t* free_state,
                           int32_t* free_state_out, int32_t* ref_cnt, int32_t num_blocks,
                           int32_t block_size, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * pkv_release_workspace_size -- bytes of device workspace that
 * pkv_release_blocks needs for num_released rows of a table of that width (0
 * for small releases). Returns a negative status on bad arguments. Needs no
 * device.
 */
int64_t pkv_release_workspace_size(int32_t num_released, int32_t max_blocks_per_req);

/*
 * The 8-bit pool
 * --------------
 * A pool of half the bytes: K and V rows as e4m3 codes, one scale byte per row.
 * The pages name no such cache; the entry points are the bf16 pool's, with the
 * same arguments, error bits and options, and `kv_scales` after `kv_cache`:
 *   kv_cache [num_blocks][2][block_size][num_kv_heads][head_dim], e4m3 codes,
 *   kv_scales[num_blocks][2][block_size][num_kv_heads], bytes; both contiguous
 *   and 16-byte aligned.
 *   value = code * 2^(scale - 127).
 * A row is the K (or V) of one token and kv head. With a = its largest magnitude,
 * e the least integer >= -117 with a <= 448 * 2^e: scale = e + 127, and each code
 * is the e4m3 number nearest to x * 2^-e, ties to even; where that would be 256
 * and e is 120 (magnitudes of 1.9375 * 2^127 and above) it is 240, for 2^128 is no
 * bf16. So a value is kept to 2^-4 of its size, or to 2^-10 * 2^e where that is more; every value that a pool
 * holds is a bf16, and rows read back and written again keep their values. A row
 * with an infinity or a NaN is held as NaN in all its elements: codes 0 and scale
 * 255 (0 * 2^128 in fp32). Scale bytes other than 10 .. 247 and 255, and the NaN
 * codes, stand in no row that was written by this library; what the calls make of
 * them is undefined, but for keys that no query row sees: those reach no output,
 * and no bit of it, whatever they hold.
 * Layout limits are the bf16 pool's; attention has two chunks' codes and the scales
 * of all kv heads in shared memory: fewer than 1800 kv heads always fit, with more
 * the call may return PKV_ERR_UNSUPPORTED.
 */

/* pkv_quant_kv_write -- pkv_paged_kv_write into the 8-bit pool: quantise each new
 * token's K and V rows and store them at its slot. Two tokens with the same slot
 * race: the row then holds undefined codes and scale. */
int32_t pkv_quant_kv_write(void* kv_cache, uint8_t* kv_scales, const void* key, const void* value,
                           int64_t key_row_stride, int64_t value_row_stride,
                           const int64_t* slot_mapping, int32_t num_tokens,
                           pkv_cache_layout layout, void* stream);

/* pkv_quant_slot_mapping_and_write -- pkv_slot_mapping_and_write into the 8-bit
 * pool: the slot mapping and the quantised write in one launch. */
int32_t pkv_quant_slot_mapping_and_write(
    void* kv_cache, uint8_t* kv_scales, const void* key, const void* value, int64_t key_row_stride,
    int64_t value_row_stride, int64_t* slot_mapping, const int32_t* block_table,
    int32_t max_blocks_per_req, const int32_t* query_start_loc, const int32_t* num_computed_tokens,
    int32_t num_reqs, int32_t num_tokens, pkv_cache_layout layout, void* stream);

/* pkv_quant_kv_read -- the inverse of pkv_quant_kv_write: key[t], value[t] = the
 * values of the rows at slot_mapping[t] (exact: they are bf16 numbers). Rows with
 * a negative slot stay as they are; so do rows with a slot outside the pool
 * (PKV_DEVERR_SLOT_RANGE). A slot may stand in the list any number of times.
 *
 * key, value    out, device bf16 [num_tokens][num_kv_heads][head_dim], row t at
 *               key + t * key_row_stride (0 = num_kv_heads * head_dim). */
int32_t pkv_quant_kv_read(void* key, void* value, int64_t key_row_stride, int64_t value_row_stride,
                          const void* kv_cache, const uint8_t* kv_scales,
                          const int64_t* slot_mapping, int32_t num_tokens, pkv_cache_layout layout,
                          void* stream);

/* pkv_quant_copy_blocks -- pkv_copy_blocks between two 8-bit pools: codes and
 * scales of every pair's block. Either pool may lie in pinned host memory. */
int32_t pkv_quant_copy_blocks(void* dst_pool, uint8_t* dst_scales, int32_t dst_num_blocks,
                              const void* src_pool, const uint8_t* src_scales,
                              int32_t src_num_blocks, const int32_t* block_pairs,
                              int32_t num_pairs, pkv_cache_layout layout, void* stream);

/*
 * pkv_quant_paged_attention -- pkv_paged_attention over the 8-bit pool: the
 * attention of the bf16 q rows over the values that the pool holds, with the same
 * options (scores, shared prefix, splits, tracing: the expansion below lies in
 * bracket [1, 2)).
 *
 * Requests of up to pkv_quant_few_rows() new tokens run on the split-KV decode
 * kernels, so a few guessed tokens of a request are checked at the cost of
 * reading its keys once. The blocks of the other requests (prompt chunks) and of
 * a shared prefix are expanded to bf16 in the workspace first, and the tensor-core
 * prefill kernel runs over those: the results of such rows are bit for bit those
 * of pkv_paged_attention over the same values.
 *
 * Precision: fp32 scores and sums. On the decode kernels a weight times V's scale is
 * an f16: 11 bits down to 2^-14 of the largest such product that a CTA meets in the
 * request, then off by 2^-25 of it at most, and zero below that. n keys together
 * lose n * 2^-25 of the largest V or less: of note where a V row is 2^14 times as
 * large as the others, in the dims that it leaves small. Outputs below
 * 2^-126 are zeros. Rows of chunks and a shared prefix: bf16 weights, and fp32 sums
 * of weight * V, which pass the largest number where V is near it.
 *
 * workspace      at least pkv_quant_attention_workspace_size() bytes, 256-byte
 *                aligned, private to this call while it runs. What lies behind the
 *                part that does not depend on chunk_keys holds the expanded
 *                blocks. If the step's chunks need more of them than fit,
 *                keys are masked out and PKV_DEVERR_CHUNK_KEYS is set.
 */
int32_t pkv_quant_paged_attention(void* out, const void* q, int64_t q_row_stride,
                                  const void* kv_cache, const uint8_t* kv_scales,
                                  const int32_t* block_table, int32_t max_blocks_per_req,
                                  const int32_t* seq_lens, const int32_t* query_start_loc,
                                  const int32_t* num_computed_tokens, int32_t num_reqs,
                                  int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len,
                                  int32_t num_q_heads, float scale, pkv_cache_layout layout,
                                  void* workspace, size_t workspace_bytes,
                                  const pkv_attention_options* options, void* stream);

/* pkv_quant_paged_attention_with_write -- pkv_paged_attention_with_write over the
 * 8-bit pool: pkv_quant_slot_mapping_and_write in the launch of the attention's
 * plan, then pkv_quant_paged_attention. */
int32_t pkv_quant_paged_attention_with_write(
    void* out, const void* q, int64_t q_row_stride, void* kv_cache, uint8_t* kv_scales,
    const void* key, const void* value, int64_t key_row_stride, int64_t value_row_stride,
    int64_t* slot_mapping, const int32_t* block_table, int32_t max_blocks_per_req,
    const int32_t* seq_lens, const int32_t* query_start_loc, const int32_t* num_computed_tokens,
    int32_t num_reqs, int32_t num_tokens, int32_t max_query_len, int32_t max_seq_len,
    int32_t num_q_heads, float scale, pkv_cache_layout layout, void* workspace,
    size_t workspace_bytes, const pkv_attention_options* options, void* stream);

/* pkv_quant_few_rows -- the most new tokens of a request that a call with this
 * max_query_len attends on the decode kernels (at least 1): max_query_len itself
 * while it times the q heads of a kv head is at most 64, else 8 / that many heads.
 * options->reserved[PKV_OPTIONS_FEW_ROWS] sets another number, from 1 to 64 / that
 * many heads (else PKV_ERR_BAD_SHAPE): for steps that hold long chunks beside
 * requests of a few tokens, whose keys the default would expand. Decodes then
 * share a kernel made for that many rows, so a larger number than the step needs
 * slows them. Needs no device. */
int32_t pkv_quant_few_rows(int32_t max_query_len, int32_t num_q_heads, int32_t num_kv_heads);

/*
 * pkv_quant_attention_workspace_size -- bytes of device workspace for
 * pkv_quant_paged_attention with up to num_reqs requests and tables of that width.
 * chunk_keys: the most cache tokens that the requests of more than
 * pkv_quant_few_rows() new tokens (or the options' number) hold between them in one step, counted in whole
 * blocks (the sum of ceil(L / block_size) * block_size); 4 * num_kv_heads *
 * head_dim bytes each. With key ranges the tokens in front of and behind those
 * that a request's rows see need not be counted. 0 is enough for steps without such
 * requests. A shared prefix of the options is counted by itself. Returns a negative
 * status on bad arguments.
 */
int64_t pkv_quant_attention_workspace_size(int32_t num_reqs, int32_t max_blocks_per_req,
                                           int32_t num_q_heads, pkv_cache_layout layout,
                                           int64_t chunk_keys,
                                           const pkv_attention_options* options);

/*
 * pkv_get_device_errors -- checked path: synchronise `stream`, then return
 * in *flags the PKV_DEVERR_* bits that kernels on the current device have set
 * since the last clear; clear them when `clear` is nonzero.
 */
int32_t pkv_get_device_errors(uint32_t* flags, int32_t clear, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H_ */
