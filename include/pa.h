/*
 * pa.h -- C ABI of libpa: single-token decode attention over a paged KV
 * cache on one GB300 (sm_103a), and what a serving step needs around it: the
 * step plan (pa_plan_step), norm, rotation and cache write
 * (pa_qk_norm_rope; pa_qk_norm_rope_axes with positions on several axes), paged
 * prefill (pa_prefill), attention with a sliding window and sinks
 * (pa_decode_window, pa_prefill_window), decode of a batch that shares a prefix
 * (pa_decode_prefix), and a cache held in 4 bits (pa_store_kv4, pa_load_kv4,
 * pa_decode_kv4).
 *
 * What the library computes.  For every sequence b < num_seqs and query head
 * h < num_heads, with G = num_heads / num_kv_heads, kvh = h / G and
 * L = seq_lens[b]:
 *
 *   l_t      = scale * dot(q[b,h,:], K[blk(t), kvh, t % block_size, :]),
 *              blk(t) = block_tables[b * max_blocks_per_seq + t / block_size]
 *   out[b,h] = sum_t exp(l_t - max l) V[blk(t), kvh, t % block_size, :]
 *              / sum_t exp(l_t - max l)                       (t < L)
 *
 * Sources (commit pages of the project "project_6"):
 *   - the paged cache and its block table, and the [blocks, kv_heads,
 *     block_size, head_dim] layout both caches use: commit 4eb83a7e
 *     "qwen3_6_scripts", paragraph "Hardware testing confirmed";
 *   - the V2 split-KV scheme (per-partition QK^T, softmax and weighted V sum
 *     into tmp_output / exp_sums / max_logits, then a cross-partition
 *     log-sum-exp reduction): same page, paragraph "Implementation
 *     (paged_attention_v2_pytorch.py)", and commit 1a4e1005 "paged_attn.py",
 *     paragraph "Architecture follows CCCL's two-pass dispatch";
 *   - the V1 single pass and the 8192-token dispatch threshold: commit
 *     1a4e1005 "paged_attn.py", change 1 "Restore V1/V2 adaptive dispatch",
 *     and commit 4eb83a7e "qwen3_6_scripts", paragraph "forward_decode: V2
 *     enabled via original heuristic";
 *   - the preallocated V2 workspace: commit 1a4e1005 "paged_attn.py",
 *     change 2 "Pre-allocate V2 intermediate tensors".
 *
 * Conventions shared by every entry point:
 *   - Every tensor pointer is a DEVICE pointer, owned by the caller, valid
 *     for the whole asynchronous execution of the call.  The library never
 *     allocates, frees, synchronises or logs (pa_read_device_status is the
 *     one call that waits on the stream, and it says so).
 *   - All work is enqueued on `stream` and returns before it runs.  The
 *     decode calls make no allocation and no host synchronisation.
 *   - Host-side checks run before anything is enqueued; a failing check
 *     returns its status and enqueues nothing.
 *   - q, k_cache, v_cache and out must be 16-byte aligned; block_tables and
 *     seq_lens 4-byte aligned; the workspace 256-byte aligned.
 *   - The caller promises 0 <= seq_lens[b] <= max_seq_len and valid block ids
 *     for every token t < seq_lens[b].  A violation is caught on the device:
 *     the offending output row is written as NaN, no out-of-range memory is
 *     touched, and (for calls given a workspace) the status word records it.
 *   - A sequence of length 0 gets an all-zero output row.
 *   - The library keeps no per-call state; calls are thread-safe.
 */
#ifndef PA_H
#define PA_H

#include <stddef.h>
#include <stdint.h>

#include <cuda_runtime_api.h>

#if defined(__GNUC__)
#define PA_API __attribute__((visibility("default")))
#else
#define PA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,         /* null pointer, bad shape or size          */
  PA_ERR_UNSUPPORTED = 2,         /* valid but not built: dtype, head_dim ... */
  PA_ERR_MISALIGNED = 3,          /* pointer alignment rule broken            */
  PA_ERR_WORKSPACE_TOO_SMALL = 4, /* workspace_bytes < pa_workspace_size()    */
  PA_ERR_CUDA = 5,                /* a CUDA launch or copy failed             */
  PA_ERR_DEVICE_TIMEOUT = 6,      /* device status: a bounded wait gave up    */
  PA_ERR_BAD_BLOCK_ID = 7,        /* device status: block id outside the pool */
  PA_ERR_BAD_SEQ_LEN = 8,         /* device status: seq_len outside 0..max    */
  PA_ERR_WORKSPACE_NOT_INIT = 9,  /* device status: pa_workspace_init missing */
  PA_ERR_NO_ROOM = 10,            /* device status: pa_plan_step refused requests:
                                     free blocks or rows ran out              */
  PA_ERR_BAD_SLOT = 11,           /* device status: slot outside the pool     */
  PA_ERR_BAD_POSITION = 12        /* device status: position outside the table */
} pa_status_t;

typedef enum pa_dtype { PA_F32 = 0, PA_BF16 = 1, PA_F16 = 2 } pa_dtype_t;

/* Flags (pa_params_t.flags). */
#define PA_FLAG_PORTABLE 1 /* use the CUDA-core kernels even where the
                              TMA / tensor-core kernels apply              */
#define PA_FLAG_SELFTEST_STALL 2 /* diagnostic: the tensor-core kernels
                              (either cache layout; prefill too) first wait
                              for an event that never happens, with a short
                              (~10 ms) bound, so their bounded-wait path
                              runs: the call's outputs become NaN and the
                              workspace status word (V2) reads
                              PA_ERR_DEVICE_TIMEOUT.  Ignored by the
                              CUDA-core kernels, which have no such waits. */
#define PA_FLAG_SPLIT_X 4 /* the caches are in the layout commit 4eb83a7e
                              "qwen3_6_scripts", paragraph "Hardware testing
                              confirmed", gives for its V1 kernel:
                                k_cache [num_blocks, num_kv_heads,
                                         head_dim / x, block_size, x]
                                v_cache [num_blocks, num_kv_heads,
                                         head_dim, block_size]
                              with x = 16 / element bytes (8 for bf16 / f16,
                              4 for f32).  Read directly, with no conversion
                              copy: for bf16 / f16 caches with block_size 16
                              or 32 and at most 8 query heads per KV head by
                              a tensor-core kernel (warp-level MMA fed by
                              ldmatrix from whole-block bulk copies; V2 in one
                              launch and V1 in clusters as on the standard
                              layout), else by the CUDA-core kernels; every
                              call accepts it. */

typedef struct pa_params {
  int32_t num_seqs;           /* B >= 0                                      */
  int32_t num_heads;          /* Hq >= 1                                     */
  int32_t num_kv_heads;       /* Hkv >= 1, divides Hq                        */
  int32_t head_dim;           /* D: 64, 128 or 256                           */
  int32_t block_size;         /* BS >= 1 tokens per physical block           */
  int32_t num_blocks;         /* NB >= 1: blocks in each cache pool          */
  int32_t max_blocks_per_seq; /* MB: row length of block_tables              */
  int32_t max_seq_len;        /* host-known upper bound of seq_lens, <= MB*BS */
  int32_t partition_size;     /* P: V2 tokens per partition, multiple of BS  */
  int32_t v1_max_seq_len;     /* pa_decode threshold, <= 0 means 8192        */
  pa_dtype_t kv_dtype;        /* element type of q, k_cache and v_cache      */
  pa_dtype_t out_dtype;       /* PA_F32, or the same type as kv_dtype        */
  float scale;                /* logit scale, usually 1/sqrt(head_dim)       */
  int32_t flags;              /* PA_FLAG_* bits, 0 by default                */
} pa_params_t;

/*
 * Tensor layouts (row-major, element type in brackets):
 *   q            [kv_dtype] [num_seqs, num_heads, head_dim]
 *   k_cache      [kv_dtype] [num_blocks, num_kv_heads, block_size, head_dim]
 *   v_cache      [kv_dtype] [num_blocks, num_kv_heads, block_size, head_dim]
 *   block_tables [int32]    [num_seqs, max_blocks_per_seq]
 *   seq_lens     [int32]    [num_seqs]
 *   out          [out_dtype][num_seqs, num_heads, head_dim]
 *
 * Workspace (V2 only), NP = ceil(max_seq_len / partition_size), each region
 * starting on a 256-byte boundary, in this order:
 *   control      1024 bytes (PA_WORKSPACE_CONTROL_BYTES), whatever the
 *                parameters: the int32 status word at offset 0, an
 *                initialisation marker at offset 4, from offset 256 the
 *                counters of the one-launch V2 step, and from offset 512 the
 *                parts' length and the queue of pa_decode_kv4
 *   max_logits   float32 [num_seqs, num_heads, NP]   m_p, natural-log units
 *   exp_sums     float32 [num_seqs, num_heads, NP]   s_p = sum exp(l_t - m_p)
 *   tmp_output   float32 [num_seqs, num_heads, NP, head_dim]
 *                o_p = sum exp(l_t - m_p) V_t / s_p
 * Only partitions p < ceil(seq_lens[b] / P) are written or read; the rest
 * may hold anything.  pa_decode_v2_partitions leaves every partition's
 * partials as defined above.  After pa_decode_v2 a sequence with a single
 * partition has no partials in the workspace.
 * The control block must be initialised once, by pa_workspace_init, before
 * the first V2 call; every V2 call leaves it ready for the next one, with
 * any parameters.
 */
#define PA_WORKSPACE_CONTROL_BYTES ((size_t)1024)

/* Bytes of workspace pa_decode_v2 / pa_decode need for these parameters
 * (0 if the parameters are invalid): the control block plus the partials.
 * Depends only on num_seqs, num_heads, head_dim, max_seq_len and
 * partition_size. */
PA_API size_t pa_workspace_size(const pa_params_t* params);

/*
 * V1: one pass per (sequence, KV head) over the whole sequence, normalised
 * straight into `out`.  No workspace: when there are fewer (sequence, KV
 * head) pairs than SMs, the tensor-core kernels (either cache layout) share
 * each pair across a thread-block cluster of up to 16 CTAs that merge their
 * partial results in distributed shared memory.
 * Source: commit 1a4e1005 "paged_attn.py", change 1 (V1 single-CTA
 * iteration); commit 4eb83a7e "qwen3_6_scripts", paragraph "V1
 * paged_attention (decode <= 8192)".
 */
PA_API pa_status_t pa_decode_v1(const pa_params_t* params, const void* q, const void* k_cache,
                         const void* v_cache, const int32_t* block_tables,
                         const int32_t* seq_lens, void* out, cudaStream_t stream);

/*
 * V2: split-KV.  Pass 1 runs per (sequence, KV-head group, partition of
 * partition_size tokens) and writes max_logits, exp_sums and tmp_output into
 * the workspace; pass 2 combines a row's partitions with weights
 * exp(m_p - max_p m_p) * s_p and writes `out`.
 * `workspace` must hold pa_workspace_size(params) bytes, its control block
 * initialised by pa_workspace_init.
 * One launch: when a tensor-core kernel (either cache layout) runs as a
 * persistent grid with at least one CTA per reduce unit (num_seqs * num_heads * head_dim / 32 units:
 * few long sequences, e.g. one 100K-token sequence), pass 2 runs in the same
 * launch.  Each CTA, after its partitions, counts itself finished in the
 * workspace; CTAs that finish once every CTA of the grid has started take
 * reduce units and run them when all are finished (no cooperative launch
 * and no wait on a CTA that has not started; the order of every sum is
 * fixed, so results are bit-identical from run to run).  Other batches and
 * the CUDA-core path use two kernels, pass 2 launched as a programmatic
 * dependent of pass 1 (pa_decode_launches() tells which).  In a workspace
 * that pa_workspace_init never initialised the one-launch step reduces
 * nothing: the status word reads PA_ERR_WORKSPACE_NOT_INIT and the rows of
 * sequences longer than one partition are NaN.
 * The V1 / V2 choice is also made per sequence inside the pass-1 launch: a
 * sequence of 1..partition_size tokens has a single partition, so pass 1
 * writes its normalised result straight into `out` (V1's contract), writes
 * no partials for it, and pass 2 skips its rows; longer sequences are split
 * and reduced.  (pa_decode_v2_partitions below always writes the partials.)
 * Source: commit 4eb83a7e "qwen3_6_scripts", paragraph "Implementation
 * (paged_attention_v2_pytorch.py)", Phase 1 and Phase 2; the per-sequence
 * choice follows the V1 / V2 tiers of commit 1a4e1005 "paged_attn.py",
 * change 1, with the partition size as the per-sequence threshold.
 */
PA_API pa_status_t pa_decode_v2(const pa_params_t* params, const void* q, const void* k_cache,
                         const void* v_cache, const int32_t* block_tables,
                         const int32_t* seq_lens, void* workspace, size_t workspace_bytes,
                         void* out, cudaStream_t stream);

/*
 * The two kernels of pa_decode_v2 as separate calls, for callers that want
 * to schedule or time them apart.  pa_decode_v2_partitions enqueues pass 1
 * and writes the workspace's partials for every partition of every
 * sequence (single-partition sequences included); pa_decode_v2_reduce
 * enqueues pass 2 (reads the workspace, writes every row of `out`) and must
 * follow pass 1 on the same stream with the same arguments.  Together they
 * give pa_decode_v2's result; pa_decode_v2 itself launches pass 2 as a
 * programmatic dependent of pass 1 and finishes single-partition sequences
 * in pass 1.
 */
PA_API pa_status_t pa_decode_v2_partitions(const pa_params_t* params, const void* q,
                                           const void* k_cache, const void* v_cache,
                                           const int32_t* block_tables, const int32_t* seq_lens,
                                           void* workspace, size_t workspace_bytes,
                                           cudaStream_t stream);
PA_API pa_status_t pa_decode_v2_reduce(const pa_params_t* params, const int32_t* seq_lens,
                                       const void* workspace, size_t workspace_bytes, void* out,
                                       cudaStream_t stream);

/*
 * Dispatch: V2 when max_seq_len > v1_max_seq_len (8192 by default), else
 * V1.  The workspace is only touched (and only required) when V2 runs.
 * Source: commit 1a4e1005 "paged_attn.py", change 1 (V2 for sequences
 * longer than 8192 tokens), and commit 4eb83a7e "qwen3_6_scripts",
 * paragraph "forward_decode: V2 enabled via original heuristic".
 */
PA_API pa_status_t pa_decode(const pa_params_t* params, const void* q, const void* k_cache,
                      const void* v_cache, const int32_t* block_tables, const int32_t* seq_lens,
                      void* workspace, size_t workspace_bytes, void* out, cudaStream_t stream);

/*
 * pa_decode_v2 for callers that cannot allocate device memory.  The pages
 * have no counterpart of this call: it exists for callers with no way to
 * call cudaMalloc or any allocator where they decode (a plugin of a host
 * runtime that owns every device allocation, a C program linking libpa
 * without torch, a real-time loop that must not stall on or fail an
 * allocation).  The caller still passes its inputs and `out`; the V2
 * workspace is instead a fixed array of PA_STATIC_WORKSPACE_BYTES (16 MiB)
 * that the library keeps in device memory, which every GPU that loads
 * libpa.so holds until the process exits.
 *   - Parameters whose pa_workspace_size() exceeds PA_STATIC_WORKSPACE_BYTES
 *     are rejected with PA_ERR_WORKSPACE_TOO_SMALL before anything is
 *     enqueued (16 MiB covers, e.g., one 24-head, head_dim-256 sequence of
 *     up to about 340K tokens at partition_size 512).
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and caches it for the current context; a new
 *     context on that device (after cudaDeviceReset, or a driver-API context
 *     the caller made current) looks it up again.  Make the first call in a
 *     context before any stream capture.
 *   - All calls on a device share the array, and it keeps the last call's
 *     contents (nothing in it needs to start at zero).  Calls that overlap on
 *     the GPU race on it: order them on one stream.
 *   - It makes no allocation of its own and calls no allocating routine.
 *   - Device-detected input errors still show as NaN output rows; the status
 *     word is not reported by this call.
 */
#define PA_STATIC_WORKSPACE_BYTES ((size_t)16 << 20)
PA_API pa_status_t pa_decode_v2_static(const pa_params_t* params, const void* q,
                                       const void* k_cache, const void* v_cache,
                                       const int32_t* block_tables, const int32_t* seq_lens,
                                       void* out, cudaStream_t stream);

/*
 * The decode step from host memory.  The per-step inputs -- q, block_tables
 * and seq_lens -- are read from HOST buffers and `out` is written to a HOST
 * buffer; k_cache, v_cache and the workspace are device memory that stays
 * resident between steps.  The call enqueues on `stream` the three
 * host-to-device copies into `staging`, the pa_decode step (V1 or V2 by the
 * same threshold) and the device-to-host copy of the result, then WAITS for
 * the stream: `out_host` is complete when it returns PA_OK.  It is therefore
 * not for use inside stream capture.
 *   staging    caller-owned device memory of pa_host_staging_size(params)
 *              bytes, 256-byte aligned; it holds the copied inputs and the
 *              result (q | block_tables | seq_lens | out, each on a 256-byte
 *              boundary) and may hold anything between calls.
 *   host buffers: page-locked memory (cudaHostAlloc / pinned tensors) makes
 *              the copies asynchronous DMA; pageable memory also works, with
 *              the copies staged by the CUDA driver.  When block_tables_host
 *              and seq_lens_host sit at the staging offsets from q_host (a
 *              host mirror of the staging layout, pa_host_staging_offsets),
 *              the three inputs move in one copy.
 * Errors: the checks of pa_decode, a null or misaligned staging buffer
 * (PA_ERR_INVALID_ARG / PA_ERR_MISALIGNED), staging_bytes too small
 * (PA_ERR_WORKSPACE_TOO_SMALL), misaligned caches (PA_ERR_MISALIGNED), all
 * before anything is enqueued; a failed copy, launch or wait gives
 * PA_ERR_CUDA.  An error found after the copies were queued is returned only
 * once the stream has finished, so no copy still uses the host buffers when
 * the call returns.
 */
PA_API size_t pa_host_staging_size(const pa_params_t* params);
/* Byte offsets within the staging layout: offsets[0] = q (0), [1] =
 * block_tables, [2] = seq_lens, [3] = out, [4] = total (= staging size).
 * PA_ERR_INVALID_ARG for invalid parameters or a null array.  Pure host
 * function. */
PA_API pa_status_t pa_host_staging_offsets(const pa_params_t* params, size_t offsets[5]);
PA_API pa_status_t pa_decode_host(const pa_params_t* params, const void* q_host,
                                  const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables_host, const int32_t* seq_lens_host,
                                  void* workspace, size_t workspace_bytes, void* staging,
                                  size_t staging_bytes, void* out_host, cudaStream_t stream);

/* Which path pa_decode takes for these parameters: 1 (V1), 2 (V2) or 0 if
 * the parameters are invalid.  Pure host function. */
PA_API int pa_decode_path(const pa_params_t* params);

/* Kernel launches one pa_decode call makes for these parameters on the
 * current device: 1 (V1, or V2 in one launch), 2 (V2 as pass 1 and a
 * dependent pass 2), 0 for invalid parameters or an empty batch.  Host
 * function; it queries the current device like pa_decode_kernel. */
PA_API int pa_decode_launches(const pa_params_t* params);

/* Which kernels the decode calls use for these parameters on the current
 * device: 2 = tensor-core kernels (bf16 / f16 caches, at most 8 query heads
 * per KV head; standard layout: TMA + tcgen05, head_dim 128 or 256 with
 * block_size 16 or 32, or head_dim 128 with block_size 64; PA_FLAG_SPLIT_X:
 * bulk copies + warp-level MMA, head_dim 64, 128 or 256 with block_size 16
 * or 32), 1 = CUDA-core kernels (every other valid case, or
 * PA_FLAG_PORTABLE), 0 = invalid parameters.  Host function; it queries the
 * current device's compute capability. */
PA_API int pa_decode_kernel(const pa_params_t* params);

/* Static description of a status code (never NULL). */
PA_API const char* pa_status_string(pa_status_t status);

/* Initialise the workspace's control block (enqueued on `stream`): zero the
 * status word and the arrival counters and write the initialisation marker
 * (the first min(workspace_bytes, PA_WORKSPACE_CONTROL_BYTES) bytes).  Call
 * once after allocating a workspace, before its first V2 call; device
 * errors then accumulate in the status word until read. */
PA_API pa_status_t pa_workspace_init(void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Diagnostic: copy the status word to *status (PA_OK or the last device
 * error recorded), WAITING for `stream` to finish, then zero it when
 * `clear` is non-zero.  Not for use inside stream capture. */
PA_API pa_status_t pa_read_device_status(const void* workspace, int32_t* status, int clear,
                                  cudaStream_t stream);

/*
 * Paged prefix prefill (chunked prefill): sequence b attends a chunk of n_b
 * new tokens to its C_b cached tokens and, causally, to the chunk itself.
 * Source: commit 1a4e1005 "paged_attn.py", opening paragraph (prefill is
 * online softmax over key tiles); commit 4eb83a7e "qwen3_6_scripts",
 * paragraphs on the prefix attention's pre-allocated m_blk / m_new / corr
 * buffers (a tile loop over the cached context, then one over the chunk),
 * "Complete rewrite of qwen3_6_scripts/paged_attn.py" item 1 (the context
 * comes from the paged cache) and "Prefill (flash_attn_func)" (causal).
 *
 *   q    [kv_dtype] [T, num_heads, head_dim]    the chunk's queries
 *   k, v [kv_dtype] [T, num_kv_heads, head_dim] the chunk's keys / values
 *   k_cache, v_cache, block_tables: as for decode; only each sequence's
 *        first ctx_lens[b] tokens are read
 *   query_start [int32] [num_seqs + 1]: sequence b owns rows
 *        query_start[b] .. query_start[b+1] - 1 of q / k / v / out
 *   ctx_lens    [int32] [num_seqs]: C_b cached tokens
 *   out  [out_dtype] [T, num_heads, head_dim]
 * Row i of sequence b (0-based in its chunk), query head h, reads KV head
 * h / (num_heads / num_kv_heads) and gives
 *   softmax(scale * q . k_j) over j = the C_b context tokens and the chunk's
 *   tokens 0..i, applied to the matching values.
 * Tensor-core kernel only: bf16 or f16, head_dim 128 (block_size 16, 32, 64)
 * or 256 (block_size 16, 32); anything else is PA_ERR_UNSUPPORTED.
 * Device-side checks: a sequence whose chunk does not satisfy
 * 0 <= n_b <= max_query_len and query_start[b+1] <= total_tokens is skipped
 * (its rows are not written); a context length outside
 * 0..min(max_ctx_len, max_blocks_per_seq * block_size), or a context block
 * id outside the pool, makes the affected rows NaN.  Asynchronous on
 * `stream`; no workspace.
 */
typedef struct pa_prefill_params {
  int32_t num_seqs;           /* B >= 0                                      */
  int32_t num_heads;          /* Hq >= 1                                     */
  int32_t num_kv_heads;       /* Hkv >= 1, divides Hq                        */
  int32_t head_dim;           /* D: 128 or 256                               */
  int32_t block_size;         /* tokens per cache block                      */
  int32_t num_blocks;         /* blocks in each cache pool                   */
  int32_t max_blocks_per_seq; /* row length of block_tables                  */
  int32_t total_tokens;       /* T: rows of q / k / v / out                  */
  int32_t max_query_len;      /* host-known bound of every n_b               */
  int32_t max_ctx_len;        /* host-known bound of every C_b               */
  pa_dtype_t kv_dtype;        /* PA_BF16 or PA_F16: q, k, v and the caches   */
  pa_dtype_t out_dtype;       /* PA_F32 or kv_dtype                          */
  float scale;                /* logit scale, usually 1/sqrt(head_dim)       */
  int32_t flags;              /* 0                                           */
} pa_prefill_params_t;

PA_API pa_status_t pa_prefill(const pa_prefill_params_t* params, const void* q, const void* k,
                              const void* v, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* query_start,
                              const int32_t* ctx_lens, void* out, cudaStream_t stream);

/*
 * The step plan: block tables, slots, positions and row starts of one serving
 * step, built on the GPU from the requests' lengths.  Request b has
 * C_b = ctx_lens[b] tokens in the cache (its first ceil(C_b / block_size)
 * table entries hold their blocks) and appends n_b = new_lens[b] tokens (1 for
 * a decode, a chunk for a prefill, 0 to sit the step out).
 *   - The blocks the new tokens need beyond those the request has are taken
 *     from the END of the free list, request by request: the i-th new block
 *     of the step is free_blocks[*free_count - 1 - i].  They are written into
 *     the request's row of block_tables; no other entry is touched.
 *   - query_start [num_seqs + 1] is the running sum of n_b, seq_lens[b] =
 *     C_b + n_b; row r = query_start[b] + i is new token i of request b, with
 *     positions[r] = *base_len + C_b + i (base_len may be null: 0; tokens of
 *     a shared prefix that the tables do not hold; the sum fits 31 bits) and
 *     slots[r] = block * block_size + (C_b + i) % block_size, the place of its
 *     key and value in the cache pool.
 *   - Rows from the step's total up to max_tokens (a padded batch) get slot
 *     -1 and position 0.  *free_left = *free_count less the blocks taken: the
 *     next step's free_count (released blocks go on the end of the list).
 *   - Requests are admitted in order: the first one whose blocks or rows do
 *     not fit, and all after it, are left as they are (no rows, no blocks,
 *     seq_lens[b] = C_b), and the status reads PA_ERR_NO_ROOM.  A request
 *     with a negative length, or with C_b + n_b > max_blocks_per_seq *
 *     block_size, gets no rows and no blocks and seq_lens[b] = max(C_b, 0)
 *     (at most the row's capacity), and the status reads PA_ERR_BAD_SEQ_LEN.
 *     A block id outside 0..num_blocks-1 (table or free list) gives its
 *     tokens slot -1 and PA_ERR_BAD_BLOCK_ID; a *free_count outside
 *     0..max_free counts as 0.
 *   - An output must not overlap an input (PA_ERR_INVALID_ARG): other CTAs
 *     still read the inputs.  Steps captured into a graph use two sets of
 *     buffers in turn.
 * status (may be null): one int32 word, as the first word of a workspace;
 * device errors are stored there and stay until read.  One launch; no
 * workspace.
 */
typedef struct pa_plan_params {
  int32_t num_seqs;           /* B >= 0                                      */
  int32_t block_size;         /* tokens per cache block                      */
  int32_t num_blocks;         /* blocks in the pool (block ids below it)     */
  int32_t max_blocks_per_seq; /* row length of block_tables                  */
  int32_t max_tokens;         /* rows of positions and slots                 */
  int32_t max_free;           /* entries of free_blocks                      */
} pa_plan_params_t;

PA_API pa_status_t pa_plan_step(const pa_plan_params_t* params, const int32_t* ctx_lens,
                                const int32_t* new_lens, const int32_t* free_blocks,
                                const int32_t* free_count, const int32_t* base_len,
                                int32_t* block_tables, int32_t* query_start, int32_t* seq_lens,
                                int32_t* positions, int64_t* slots, int32_t* free_left,
                                int32_t* status, cudaStream_t stream);

/*
 * Norm of each query and key head, rotation by position, and the write of
 * keys and values into the paged cache, in one pass over the projections.
 * For row t and head h, x the head_dim elements of q[t,h] (or k[t,h]):
 *   y = x * (1 / sqrt(mean(x^2) + eps)) * (weight + weight_offset)
 * (no norm where the weight is null), then the first rotary_dim elements are
 * rotated in pairs (a, b) by the row's angles, c_j = cos_sin[pos][j] and
 * s_j = cos_sin[pos][rotary_dim / 2 + j]:
 *   (a, b) -> (a c_j - b s_j, b c_j + a s_j),
 * pair j being elements (j, j + rotary_dim / 2), or (2j, 2j + 1) with
 * PA_ROPE_INTERLEAVED.  Sums and products are float32, rounded once.
 *   q [T, num_heads, head_dim], k, v [T, num_kv_heads, head_dim]: rows
 *        q_stride / k_stride / v_stride elements apart (slices of one fused
 *        projection), heads contiguous within a row; 16-byte aligned rows
 *   q_out [T, num_heads, head_dim], contiguous
 *   k_out, v_out [T, num_kv_heads, head_dim], contiguous, may be null: the
 *        normed and rotated keys, and the values, as pa_prefill takes them
 *   k_cache, v_cache: the pools (standard layout, or PA_FLAG_SPLIT_X); row t
 *        is stored at slot slots[t] = block * block_size + place.  Both may
 *        be null (slots then only marks padding).
 *   q_weight, k_weight [head_dim], element type as q; both null: no norm
 *   cos_sin float32 [max_position, rotary_dim]
 *   positions int32 [T], slots int64 [T]
 * A row with slot -1 is padding: nothing of it is written.  With caches a slot
 * outside the pool (below -1, or past num_blocks * block_size) writes no cache
 * and reads PA_ERR_BAD_SLOT in the status; a position outside
 * 0..max_position-1 makes the row's q_out and k_out NaN, writes no cache and
 * reads PA_ERR_BAD_POSITION.  Rows must have distinct slots: where two rows
 * share one, what it holds afterwards is some mix of the two.
 * No output may overlap an input or another output (PA_ERR_INVALID_ARG), but
 * q_out may be q itself where q is contiguous, and so k_out and v_out.
 * rotary_dim is a multiple of 16, at most head_dim (0: no rotation).  Without
 * rows (num_tokens 0) no address is looked at: each may be null, as those of empty
 * tensors are.  One launch; no workspace; status as for pa_plan_step.
 */
#define PA_ROPE_INTERLEAVED 256 /* pa_rope_params_t.flags, beside PA_FLAG_SPLIT_X */
typedef struct pa_rope_params {
  int32_t num_tokens;   /* T >= 0                                            */
  int32_t num_heads;    /* Hq >= 1                                           */
  int32_t num_kv_heads; /* Hkv >= 1                                          */
  int32_t head_dim;     /* D: 64, 128 or 256                                 */
  int32_t block_size;   /* tokens per cache block                            */
  int32_t num_blocks;   /* blocks in each cache pool                         */
  int32_t rotary_dim;   /* elements rotated                                  */
  int32_t max_position; /* rows of cos_sin                                   */
  int64_t q_stride;     /* elements from one row of q to the next            */
  int64_t k_stride;
  int64_t v_stride;
  pa_dtype_t dtype;     /* q, k, v, weights, caches and outputs              */
  int32_t flags;        /* PA_ROPE_INTERLEAVED, PA_FLAG_SPLIT_X              */
  float eps;
  float weight_offset;  /* added to the weights (0, or 1 for weights around 0) */
} pa_rope_params_t;

PA_API pa_status_t pa_qk_norm_rope(const pa_rope_params_t* params, const void* q, const void* k,
                                   const void* v, const void* q_weight, const void* k_weight,
                                   const float* cos_sin, const int32_t* positions,
                                   const int64_t* slots, void* q_out, void* k_out, void* v_out,
                                   void* k_cache, void* v_cache, int32_t* status,
                                   cudaStream_t stream);

/*
 * The same with several positions a row, one for each axis of an image or a video
 * (time, height, width): pair j of the rotation turns by the angle of its own
 * axis' position,
 *   c_j = cos_sin[positions[axis_of[j]][t]][j], s_j likewise.
 *   positions int32 [num_axes, T]; text has the same position on every axis
 * A row with a position outside 0..max_position-1 on any axis is handled as
 * pa_qk_norm_rope handles its one position.  Everything else is as there; with
 * one axis so are the results.
 */
#define PA_ROPE_MAX_AXES 4
#define PA_ROPE_MAX_PAIRS 128
typedef struct pa_rope_axes {
  int32_t num_axes;                   /* 1..PA_ROPE_MAX_AXES                   */
  uint8_t axis_of[PA_ROPE_MAX_PAIRS]; /* axis of pair j < rotary_dim / 2       */
} pa_rope_axes_t;

PA_API pa_status_t pa_qk_norm_rope_axes(const pa_rope_params_t* params,
                                        const pa_rope_axes_t* axes, const void* q, const void* k,
                                        const void* v, const void* q_weight,
                                        const void* k_weight, const float* cos_sin,
                                        const int32_t* positions, const int64_t* slots,
                                        void* q_out, void* k_out, void* v_out, void* k_cache,
                                        void* v_cache, int32_t* status, cudaStream_t stream);

/*
 * Attention with a sliding window and sinks.  A query at position p (0-based)
 * sees token t <= p when t < num_sinks (the sequence's first tokens, which stay
 * visible) or t > p - window (the last `window` tokens, itself included).
 * Tokens outside are not read: block-table entries of blocks that hold no
 * visible token may say anything (blocks given back to the pool).
 */
typedef struct pa_window {
  int32_t window;    /* >= 1                                                 */
  int32_t num_sinks; /* >= 0                                                 */
} pa_window_t;

/*
 * Decode: the step of pa_decode (same tensors, layouts, flags and checks; the
 * query sits at position seq_lens[b] - 1) over the visible tokens.  The
 * workspace holds pa_window_workspace_size() bytes, its control block
 * initialised by pa_workspace_init; partition_size (a multiple of block_size,
 * as for pa_decode_v2) is the tokens of one partial of a row where there are
 * many sequences; for few the tensor-core kernel's split is chosen to fill
 * the GPU.  A workspace for some num_seqs and max_seq_len serves smaller ones.
 * Tensor-core kernel where pa_decode_kernel() says 2 and the layout is the
 * standard one, else CUDA cores.  v1_max_seq_len is not used.  What the pools hold for
 * invisible tokens does not matter (NaN included).
 */
PA_API size_t pa_window_workspace_size(const pa_params_t* params, const pa_window_t* window);
PA_API pa_status_t pa_decode_window(const pa_params_t* params, const pa_window_t* window,
                                    const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, const int32_t* seq_lens,
                                    void* workspace, size_t workspace_bytes, void* out,
                                    cudaStream_t stream);

/*
 * Prefill: the chunk of pa_prefill (same tensors and device-side checks) with
 * the same mask; row i of sequence b sits at position ctx_lens[b] + i.  Every
 * dtype, head_dim (64, 128, 256) and block size the decode calls take:
 * tensor-core kernel for bf16 / f16, head_dim 128 (block_size 16, 32, 64) or
 * 256 (16, 32) and at most 64 query heads per KV head, else CUDA cores
 * (flags: PA_FLAG_PORTABLE, PA_FLAG_SPLIT_X for the caches,
 * PA_FLAG_SELFTEST_STALL).  Of the tokens that at least one row of the call
 * sees, values must be finite (a weight of zero times infinity is NaN).
 * The call has no status word: what the device-side checks find shows as NaN
 * rows, or as rows that are not written, only.
 * Rounding: logits, maxima, sums and accumulators are float32.  The tensor-core
 * kernel rounds each softmax weight once to the element type before the product
 * with the values, as pa_prefill does (half a step: 2^-8 of the weight for bf16,
 * 2^-11 for f16, and for f16 2^-32 of the row's largest); the sum takes it
 * unrounded.  The CUDA-core kernel (PA_FLAG_PORTABLE) keeps it in float32.
 */
PA_API pa_status_t pa_prefill_window(const pa_prefill_params_t* params, const pa_window_t* window,
                                     const void* q, const void* k, const void* v,
                                     const void* k_cache, const void* v_cache,
                                     const int32_t* block_tables, const int32_t* query_start,
                                     const int32_t* ctx_lens, void* out, cudaStream_t stream);

/*
 * Decode of a batch that shares a prefix.  Every sequence attends to the
 * *prefix_len tokens of one shared prefix (blocks prefix_blocks[0 ..], the
 * last one possibly part full) and then to its own seq_lens[b] tokens (blocks
 * block_tables[b], which hold nothing of the prefix):
 *   out[b,h] = softmax over both lists of scale * q[b,h] . k, applied to v.
 * On the tensor cores the prefix is read once for all sequences and heads of a
 * KV group, as one matrix product over the rows (b, h); the CUDA-core kernel
 * reads it for each sequence.  The own tokens go through the paged decode pass, or
 * with the join through a kernel for many short lists; the last kernel joins the
 * partial results.
 *   prefix_blocks [int32] [max_prefix_blocks], prefix_len [int32] [1], on the
 *   device; seq_lens[b] in 0..max_seq_len, and both lists may be empty (a row
 *   with no token at all is zeros).
 * A prefix length outside 0..max_prefix_len, or a prefix block id outside the
 * pool, makes every row NaN; a sequence's own bad length or block id its rows.
 * The workspace's status word reads PA_ERR_BAD_SEQ_LEN or PA_ERR_BAD_BLOCK_ID,
 * also where a bound is 0.
 * workspace: pa_prefix_workspace_size() bytes, initialised once by
 * pa_workspace_init; one for some num_seqs, max_seq_len and max_prefix_len
 * serves smaller ones.  Tensor-core kernel for the prefix with the shapes that
 * pa_prefill_window's has, else CUDA cores.
 * Rounding: the tensor-core prefix pass rounds the weights as pa_prefill_window's
 * kernel does, so the prefix's part of the result is off by about half a step of
 * the element type where pa_decode, which keeps some 16 bits of each weight, is
 * not: with a 16-bit output about 1.3 times pa_decode's error.  The own tokens keep
 * 16 bits; PA_FLAG_PORTABLE keeps float32 weights throughout.
 */
typedef struct pa_prefix {
  int32_t max_prefix_len;    /* host-known bound of *prefix_len              */
  int32_t max_prefix_blocks; /* entries of prefix_blocks                     */
} pa_prefix_t;

PA_API size_t pa_prefix_workspace_size(const pa_params_t* params, const pa_prefix_t* prefix);
PA_API pa_status_t pa_decode_prefix(const pa_params_t* params, const pa_prefix_t* prefix,
                                    const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* prefix_blocks, const int32_t* prefix_len,
                                    const int32_t* block_tables, const int32_t* seq_lens,
                                    void* workspace, size_t workspace_bytes, void* out,
                                    cudaStream_t stream);

/*
 * The paged cache held in 4 bits.  A pool of num_blocks pages holds, for keys and
 * for values each,
 *   codes  [num_blocks, num_kv_heads, block_size, head_dim / 2] bytes: element 2i
 *          of a head row is the low half of byte i, element 2i + 1 the high half;
 *   scales [num_blocks, num_kv_heads, block_size, head_dim / group_size, 2] of the
 *          model's element type: a scale and a minimum for each group of
 *          group_size (32, 64 or 128, dividing head_dim) elements of a head row.
 * A code c in 0..15 stands for the value c * scale + minimum.  dtype is the type of
 * the scales, of the rows stored and of the queries: float32, bf16 or f16; head_dim
 * is 64, 128 or 256.  Codes and scales are 16-byte aligned.  Block tables, lengths
 * and slots are those of the other calls (pa_plan_step's).
 *
 * pa_store_kv4 writes the keys and values of T rows into such a pool.  For each
 * group of a head row x, m = min x, s = (max x - m) / 15 rounded to the element
 * type, and each element's code is (x - m) / s rounded to the nearest whole number
 * (halves to even), at most 15, or 0 where s is 0.  A group with an element that is
 * not finite, or a range past float32, gets NaN for both and reads back as NaN.  The
 * rounding of s moves code 15's value by up to half a step, relative, of the group's range:
 * where it passes the type's largest number it reads back as infinity.
 *   k, v [T, num_kv_heads, head_dim]: rows k_stride / v_stride elements apart,
 *        heads contiguous within a row; 16-byte aligned rows
 *   slots int64 [T]: slot block * block_size + place; -1 is padding (nothing of the
 *        row is written); another slot outside the pool writes no cache and reads
 *        PA_ERR_BAD_SLOT in the status.  Rows must have distinct slots.
 *   k_out, v_out [T, num_kv_heads, head_dim], contiguous, may be null: the values
 *        that the codes stand for, rounded to the element type -- the chunk's keys
 *        and values for pa_prefill, as later steps will see them.
 * No output may overlap an input or another output (PA_ERR_INVALID_ARG), but k_out
 * may be k itself where k is contiguous, and so v_out.  One launch; no workspace;
 * status as for pa_plan_step.
 */
typedef struct pa_store_kv4_params {
  int32_t num_tokens;   /* T >= 0                                            */
  int32_t num_kv_heads; /* Hkv >= 1                                          */
  int32_t head_dim;     /* D: 64, 128 or 256                                 */
  int32_t block_size;   /* tokens per page                                   */
  int32_t num_blocks;   /* pages in the pool                                 */
  int32_t group_size;   /* 32, 64 or 128, divides D                          */
  int64_t k_stride;     /* elements from one row of k to the next            */
  int64_t v_stride;
  pa_dtype_t dtype;     /* k, v, k_out, v_out and the scales                 */
} pa_store_kv4_params_t;

PA_API pa_status_t pa_store_kv4(const pa_store_kv4_params_t* params, const void* k, const void* v,
                                const int64_t* slots, void* k_codes, void* v_codes,
                                void* k_scales, void* v_scales, void* k_out, void* v_out,
                                int32_t* status, cudaStream_t stream);

/*
 * pa_load_kv4 widens pages of the 4-bit pool into pages of the element type
 * (the standard layout [num_out_blocks, num_kv_heads, block_size, head_dim]), so that
 * pa_prefill and pa_prefill_window can read a context that is held in 4 bits:
 * for each sequence b and j < ceil(seq_lens[b] / block_size), page
 * block_tables[b][j] becomes page out_tables[b][j] of k_out and v_out, each value
 * rounded once.  Whole pages are written, places past the sequence's end included;
 * no other page is touched.  Pages of out_tables must be distinct.
 * A length outside 0..max_seq_len leaves the sequence out and reads
 * PA_ERR_BAD_SEQ_LEN in the status; a page outside its pool reads
 * PA_ERR_BAD_BLOCK_ID, and the page of out_tables becomes NaN (a bad source) or none
 * is written (a bad destination).  No output may overlap an input or another output.
 * One launch; no workspace; status as for pa_plan_step.
 */
typedef struct pa_load_kv4_params {
  int32_t num_seqs;               /* B >= 0                                  */
  int32_t num_kv_heads;           /* Hkv >= 1                                */
  int32_t head_dim;               /* D: 64, 128 or 256                       */
  int32_t block_size;             /* tokens per page, of both pools          */
  int32_t num_blocks;             /* pages in the 4-bit pool                 */
  int32_t max_blocks_per_seq;     /* row length of block_tables              */
  int32_t num_out_blocks;         /* pages in k_out and v_out                */
  int32_t max_out_blocks_per_seq; /* row length of out_tables                */
  int32_t max_seq_len;            /* host-known bound of every seq_lens[b]   */
  int32_t group_size;             /* 32, 64 or 128, divides D                */
  pa_dtype_t dtype;               /* the scales, k_out and v_out             */
} pa_load_kv4_params_t;

PA_API pa_status_t pa_load_kv4(const pa_load_kv4_params_t* params, const void* k_codes,
                               const void* v_codes, const void* k_scales, const void* v_scales,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               const int32_t* out_tables, void* k_out, void* v_out,
                               int32_t* status, cudaStream_t stream);

/*
 * Decode over the 4-bit cache: the step of pa_decode (same q, tables, lengths, out
 * and checks; kv_dtype is the type of q and of the scales) with keys and values
 * c * scale + minimum.  Scales and minima of visible tokens are finite, or NaN,
 * which makes the rows that see them NaN; what the pools hold elsewhere does not
 * matter.  The workspace holds pa_kv4_workspace_size() bytes, its control block
 * initialised by pa_workspace_init; it serves one call at a time, and one for some
 * num_seqs and max_seq_len serves smaller ones.  partition_size (>= 1) bounds the slots
 * for partials where there are many sequences: a row's parts are that long, in whole
 * tiles of 64 tokens, or longer, up to 2^17 tokens.  The tensor-core kernel chooses their length on the
 * device, from the lengths of the call, so results depend on the batch by what the order
 * of float32 sums does.  Where max_seq_len is at most 131072 / head_dim (half of that where
 * num_seqs * num_kv_heads * ceil(num_heads / num_kv_heads / 8) is at most 19, twice where
 * it is above 1824), rows have one part and the call is one launch.
 * v1_max_seq_len is not used; flags: PA_FLAG_PORTABLE.
 * Tensor-core kernel for bf16 and f16, CUDA cores for float32 and PA_FLAG_PORTABLE.
 * Rounding: codes, scales and minima are used as they are; logits, maxima, sums and
 * accumulators are float32.  With weights taken beside the row's largest, as 1, the
 * tensor-core kernel rounds the product of a weight and a value's scale once, to 11 bits
 * (half a step, 2^-11 of it, or 2^-35 of the largest scale of that group in the sequence where
 * that is more), where it multiplies codes around the middle of the group, at most 8 steps
 * from it; and the weights that meet the minima to 2^-17 (bf16) or 2^-22 (f16, or 2^-33 of a
 * weight of 1).  So a token with scales up to 2^24 times another's costs that one no bits,
 * however little weight it has.  Elements of a query head are whole to 2^-24 of its largest,
 * below that off by up to 2^-35 of it.  Queries of 2^116 and more make their row NaN, and
 * the weighted sum of values is taken times up to 2^12: values whose sum over the row passes
 * 2^115 overflow.  The CUDA-core kernel keeps float32.
 */
typedef struct pa_kv4 {
  int32_t group_size; /* 32, 64 or 128, divides head_dim                     */
} pa_kv4_t;

PA_API size_t pa_kv4_workspace_size(const pa_params_t* params, const pa_kv4_t* kv4);
PA_API pa_status_t pa_decode_kv4(const pa_params_t* params, const pa_kv4_t* kv4, const void* q,
                                 const void* k_codes, const void* v_codes, const void* k_scales,
                                 const void* v_scales, const int32_t* block_tables,
                                 const int32_t* seq_lens, void* workspace,
                                 size_t workspace_bytes, void* out, cudaStream_t stream);

/* ABI version: major * 10000 + minor * 100 + patch.  200: the serving-step calls; 300:
 * pa_qk_norm_rope_axes and the calls on the 4-bit cache. */
PA_API int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H */
