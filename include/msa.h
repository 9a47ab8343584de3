/*
 * msa.h -- C ABI of the GB300 (sm_103a) MSA block-sparse top-k attention backward.
 *
 * The operation is the backward pass of MiniMax-M3 MSA attention as stated on
 * the NVIDIA NeMo AutoModel API pages for minimax_m3_vl: every query chunk of
 * C = 8 tokens and each index head attends only to its selected top-k key
 * blocks of B = 64 keys, causally within the packed documents of cu_seqlens,
 * with G = 16 query heads sharing one index/KV head; the pass returns dQ, dK
 * and dV in bf16 ("msa_backward_sm100" page, module docstring and
 * run_backward; "msa_schedule" page, MSABackwardSchedule).
 *
 * Conventions shared by every call:
 *  - Every pointer named "device" is CUDA device memory owned by the caller.
 *    The library allocates nothing, never synchronises and keeps no state
 *    between calls except memoised device queries (SM count, capability).
 *  - Calls are asynchronous and ordered on the given stream (a cudaStream_t
 *    passed as void*; NULL is the legacy default stream).
 *  - Tensors are row-major THD: [tokens, heads, head_dim] with head_dim
 *    contiguous, the view the pages' _head_major helper describes.  bf16
 *    tensors are passed as uint16_t bit patterns.  Every pointer must be
 *    16-byte aligned (the pages' _operand helper).
 *  - The return value reports errors detectable on the host.  Errors found on
 *    the device (capacity, invalid selection, timeout) are written to the
 *    caller's device word *d_status with the first error winning; the caller
 *    sets it to 0 before a sequence of calls and reads it after a sync.  Each
 *    kernel returns without touching its outputs if *d_status is already
 *    non-zero, so tables from a failed build are never consumed.
 */
#ifndef MSA_H_
#define MSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes.  The pages raise TypeError/ValueError on a malformed schedule
 * ("msa_schedule" page, MSABackwardSchedule, Raises) and NotImplementedError
 * on a device that is not the one the kernels are built for ("kernels" page,
 * require_sm100); here both become integer codes. */
enum {
  MSA_OK = 0,
  MSA_ERR_INVALID_ARGUMENT = 1,   /* null / misaligned pointer, bad size or count        */
  MSA_ERR_UNSUPPORTED_DEVICE = 2, /* compute capability is not 10.3 (sm_103a build)     */
  MSA_ERR_UNSUPPORTED_SHAPE = 3,  /* a shape the kernels are not built for               */
  MSA_ERR_CAPACITY = 4,           /* edge_cap or task_cap too small (device-detected)    */
  MSA_ERR_INVALID_SELECTION = 5,  /* sel entry out of range, non-causal or repeated      */
  MSA_ERR_TIMEOUT = 6,            /* a bounded device wait expired                       */
  MSA_ERR_CUDA = 7,               /* a CUDA launch or runtime call failed                */
  MSA_ERR_INVALID_DOCUMENTS = 8,  /* cu_seqlens / kv_doc_starts inconsistent (device)    */
  MSA_ERR_SCRATCH_TOO_SMALL = 9,  /* problem exceeds the no-allocation scratch array     */
  MSA_ERR_INVALID_CACHE = 10      /* cache tables, lengths or slots inconsistent (device) */
};

/* Problem description.  Mirrors run_backward's tensor contract
 * ("msa_backward_sm100" page, run_backward parameters) and the schedule's
 * cu_seqlens / document_workspace_starts ("msa_schedule" page).
 *
 * num_docs        N >= 1 documents packed along the token axis.
 * total_tokens    T = cu_seqlens[N].
 * cu_seqlens      device int32 [N+1]; cu[0] = 0, strictly increasing.
 * kv_doc_starts   device int32 [N]; K/V row of each document's first key.
 *                 Equal to cu_seqlens[0..N) for compact K/V; a multiple of
 *                 128 per document for the pages' aligned workspace.  Ranges
 *                 [kv_doc_starts[d], kv_doc_starts[d] + len_d) must increase
 *                 with d and not overlap.  K/V rows outside every document
 *                 must hold finite values; their gradients are written as 0.
 * kv_rows         W, rows of the K/V workspace (W = T for compact K/V).
 * num_q_heads     Hq; num_index_heads = num_kv_heads = Hq / 16.
 * head_dim        128.   block_size 64.   query_chunk 8.
 * topk            K, 1 <= K <= 32, slots per (index head, query chunk).
 * num_blocks      NB = sum_d ceil(len_d / block_size) (host copy, for sizing).
 * num_chunks      NC = sum_d ceil(len_d / query_chunk).
 * softmax_scale   scale applied to q.k (the pages use head_dim ** -0.5).
 */
typedef struct {
  int32_t num_docs;
  int32_t total_tokens;
  const int32_t* cu_seqlens;
  const int32_t* kv_doc_starts;
  int32_t kv_rows;
  int32_t num_q_heads;
  int32_t num_index_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t query_chunk;
  int32_t topk;
  int32_t num_blocks;
  int32_t num_chunks;
  float softmax_scale;
} msa_problem;

/* Columns of a task_meta row: the pages' scheduler_metadata column order
 * (index_head, row_linear, q_begin, q_count, document_ordinal,
 * document_local_kblock) ("msa_schedule" page, MSABackwardSchedule).
 * q_begin is the CSR offset of the task's first query entry. */
enum { MSA_TASK_META_COLS = 6 };

/* Layout of the int32 walk descriptor written by msa_build_tasks: the CTA
 * walk rule of the "msa_schedule" page (rows_per_cta, chunk_map).
 * walk[MSA_WALK_ROWS] rows (tasks); [MSA_WALK_ROWS_PER_CTA] R (4 below 2400
 * rows, else 64); [MSA_WALK_FULL] full units of R rows; [MSA_WALK_TAIL] tail
 * rows; [MSA_WALK_GRID] units = full + min(tail, num_sms); [MSA_WALK_SMS]. */
enum {
  MSA_WALK_ROWS = 0, MSA_WALK_ROWS_PER_CTA = 1, MSA_WALK_FULL = 2, MSA_WALK_TAIL = 3,
  MSA_WALK_GRID = 4, MSA_WALK_SMS = 5, MSA_WALK_LEN = 8
};

/* Bytes of device workspace one sequence msa_build_k2q -> msa_build_tasks ->
 * msa_bwd needs (the calls may share one buffer, used in stream order).
 * Returns 0 if the problem is invalid. */
size_t msa_workspace_bytes(const msa_problem* p, int64_t edge_cap, int64_t task_cap,
                           int32_t task_tile_chunks);
/* msa_workspace_bytes for a backward run with options (MSA_BWD_DQ_FP32 adds
 * an fp32 dQ accumulator of T * Hq * 128 * 4 bytes).  Returns 0 for an
 * invalid problem or an unknown option bit. */
size_t msa_workspace_bytes_opts(const msa_problem* p, int64_t edge_cap, int64_t task_cap,
                                int32_t task_tile_chunks, uint32_t options);

/* Key-block -> query CSR ("msa_bindings" page, build_k2q_csr;
 * "msa_schedule" page, row_ptr and q_indices).
 *
 * sel        device int32 [Hi, NC, K]: for index head hi and global query
 *            chunk g (document-major numbering), the document-local key
 *            blocks the chunk attends; -1 marks an empty slot (any slot).
 *            Valid entries are distinct and causal: b * block_size <= the
 *            chunk's first query position; otherwise *d_status =
 *            MSA_ERR_INVALID_SELECTION.
 * row_ptr    device int32 [Hi, NB+1] out: row r = blk_off[d] + b of head hi
 *            holds q_indices[hi][row_ptr[hi][r] .. row_ptr[hi][r+1]).
 * q_indices  device int32 [Hi, edge_cap] out: document-local query positions
 *            of each row, ascending.  Entries past a head's last row are
 *            left untouched.
 * edge_cap   capacity per head; too small -> *d_status = MSA_ERR_CAPACITY.
 * The result is deterministic (bit-identical on every run).
 */
int msa_build_k2q(const msa_problem* p, const int32_t* sel, int32_t* row_ptr, int32_t* q_indices,
                  int64_t edge_cap, int32_t* d_status, void* ws, size_t ws_bytes, void* stream);

/* msa_build_k2q for callers that cannot allocate device memory.  The pages
 * have no counterpart: this entry point exists for library users, not for the
 * method.  Some callers may not call cudaMalloc at all: a host framework whose
 * caching allocator or fixed memory pool owns all device memory, or a latency-
 * sensitive path that cannot afford cudaMalloc's implicit synchronisation.
 * They still pass sel, row_ptr, q_indices and d_status, exactly as for
 * msa_build_k2q; the build's scratch (document offsets, per-group counts and
 * row totals) lives in one array of MSA_NOALLOC_SCRATCH_BYTES that the library
 * holds on every GPU that loads it, until the process exits.
 *  - The scratch a problem needs is about 8 (N+1) + 4 Hi NB (G+1) bytes, with
 *    G = ceil(NC / S) scatter groups of S = max(64, ceil(NC / 128)) query
 *    chunks (so G <= 128); a problem needing more is rejected with
 *    MSA_ERR_SCRATCH_TOO_SMALL before anything is launched.  One document of
 *    131,072 tokens with 8 index heads needs about 8.5 MB.
 *  - The first call on a device looks up the array's device address (a
 *    runtime query made once per device, with that device current); make that
 *    first call before any stream capture begins.  The address is kept with
 *    the ID of the CUDA context it belongs to: after cudaDeviceReset (a new
 *    context, where the array may sit elsewhere) the next call looks it up
 *    again, and that call too should come before any capture.
 *  - Every call uses the same array and it keeps what the last call left
 *    there; the build overwrites all of it before reading, so nothing in it
 *    needs to start at zero.  Calls whose kernels overlap on the GPU (other
 *    streams, other host threads) race on the array and must be serialised by
 *    the caller.
 * It allocates nothing and returns the same codes as msa_build_k2q. */
#define MSA_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
int msa_build_k2q_noalloc(const msa_problem* p, const int32_t* sel, int32_t* row_ptr,
                          int32_t* q_indices, int64_t edge_cap, int32_t* d_status, void* stream);

/* Task rows and CTA walk of the KV-parallel backward ("msa_backward_sm100"
 * page, module docstring: task rows of 8 queries x 16 heads bucketed by
 * (batch, index_head, key_block); "msa_schedule" page, chunk_map,
 * rows_per_cta, grid_launch_bound).
 *
 * Each CSR row is cut into consecutive groups of query_chunk entries; a group
 * is one task (one query chunk against one key block).  Tasks are ordered by
 * index head, then query tile (global chunk / task_tile_chunks; 0 = a single
 * tile), then key-block row, then CSR offset.
 * task_meta   device int32 [task_cap, 6] out (MSA_TASK_META_COLS).
 * task_q_rows device int32 [task_cap, query_chunk] out: compact token row of
 *             each query slot, -1 past q_count.  Slots of one task are
 *             consecutive tokens of one chunk.
 * task_q_pos  device int32 [task_cap, query_chunk] out: document-local
 *             position of each slot, -1 past q_count.
 * walk        device int32 [MSA_WALK_LEN] out.
 * num_sms     SMs the walk is sized for; 0 = the current device's count.
 * Too many tasks for task_cap -> *d_status = MSA_ERR_CAPACITY.
 */
int msa_build_tasks(const msa_problem* p, const int32_t* row_ptr, const int32_t* q_indices,
                    int64_t edge_cap, int32_t task_tile_chunks, int32_t* task_meta,
                    int32_t* task_q_rows, int32_t* task_q_pos, int32_t* walk, int64_t task_cap,
                    int32_t num_sms, int32_t* d_status, void* ws, size_t ws_bytes, void* stream);

/* The backward pass ("msa_backward_sm100" page, run_backward): preprocess
 * D = rowsum(dO * O), the KV-parallel tcgen05 kernel over the task rows, and
 * the postprocess cast of the fp32 accumulators to bf16.
 *
 * q, o, dout  device bf16 [T, Hq, 128]; lse device fp32 [T, Hq] natural-log
 *             log-sum-exp of the forward.
 * k, v        device bf16 [W, Hkv, 128].
 * task_*      tables written by msa_build_tasks for this problem.
 * dq          device bf16 [T, Hq, 128] out.
 * dk, dv      device bf16 [W, Hkv, 128] out; rows outside every document 0.
 * ws          workspace of at least msa_workspace_bytes() bytes.
 */
int msa_bwd(const msa_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
            const uint16_t* o, const uint16_t* dout, const float* lse, const int32_t* task_meta,
            const int32_t* task_q_rows, const int32_t* task_q_pos, const int32_t* walk,
            int64_t task_cap, uint16_t* dq, uint16_t* dk, uint16_t* dv, int32_t* d_status,
            void* ws, size_t ws_bytes, void* stream);

/* msa_bwd split at its kernel boundaries, for callers that interleave their
 * own work or time the stages: stages is a mask of MSA_STAGE_* run in order
 * preprocess -> main -> postprocess on the stream.  msa_bwd is
 * stages = MSA_STAGE_ALL.  The stages communicate through ws, so a later
 * stage must see the same ws, tables and inputs as the earlier ones. */
enum { MSA_STAGE_PREPROCESS = 1, MSA_STAGE_MAIN = 2, MSA_STAGE_POSTPROCESS = 4, MSA_STAGE_ALL = 7 };
/* Option bit of the same mask: accumulate dQ in fp32.  By default each
 * task's fp32 dQ (over its 64 keys) is rounded to bf16 and reduce-added into
 * the bf16 dQ output, as the pages' bf16 dQ pool is ("msa_schedule" page,
 * the bf16x2 dQ pool; "msa_backward_sm100" page, dQ atomics), so a row of dQ
 * takes one bf16 rounding per task that feeds it.  With MSA_BWD_DQ_FP32 the
 * tasks reduce-add fp32 tiles into an fp32 buffer in ws (twice the reduce
 * traffic), which the postprocess rounds once to bf16.  ws must then hold
 * msa_workspace_bytes_opts(..., MSA_BWD_DQ_FP32) bytes, and every stage of
 * one backward must be called with the same option. */
enum { MSA_BWD_DQ_FP32 = 8 };
/* Self-test bit of the same mask (no counterpart in the pages; outputs are
 * not to be used): the main stage runs with its reduce warps idle, so the
 * hand-offs that wait for them (the task-info ring, the dQ buffers) run out
 * their 2 s bound, every role of the kernel aborts, in-flight copies are
 * waited for, and *d_status reads MSA_ERR_TIMEOUT.  The context stays usable.
 * Not combinable with MSA_BWD_DQ_FP32 (MSA_ERR_INVALID_ARGUMENT). */
enum { MSA_BWD_SELFTEST_HOLD_REDUCE = 16 };
int msa_bwd_staged(const msa_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                   const uint16_t* o, const uint16_t* dout, const float* lse, const int32_t* task_meta,
                   const int32_t* task_q_rows, const int32_t* task_q_pos, const int32_t* walk,
                   int64_t task_cap, uint16_t* dq, uint16_t* dk, uint16_t* dv, int32_t* d_status,
                   void* ws, size_t ws_bytes, void* stream, uint32_t stages);

/* The forward pass that produces O and LSE from the same selection
 * ("msa_bindings" page, sparse_atten_func, the flat forward): for each query
 * row, softmax(scale * q k^T) over the keys of its chunk's selected blocks
 * that precede or equal it, times V.  One pass with an online softmax; P is
 * rounded to bf16 for the P V product, everything else accumulates in fp32.
 * q     device bf16 [T, Hq, 128];  k, v device bf16 [W, Hkv, 128].
 * sel   device int32 [Hi, NC, K], as for msa_build_k2q (validated there,
 *       not here: call the forward with a selection the CSR build accepted).
 * o     device bf16 [T, Hq, 128] out;  lse device fp32 [T, Hq] out (natural
 *       log; -inf for a query that attends no key, whose O is 0).
 * ws    device workspace of at least 8 * (num_docs + 1) bytes rounded up to
 *       256 (msa_workspace_bytes() is always enough); caller-owned.
 * Returns MSA_ERR_INVALID_ARGUMENT for a null or misaligned pointer or a short
 * ws, MSA_ERR_CUDA if a launch fails; a device wait that exceeds its bound
 * writes MSA_ERR_TIMEOUT to *d_status.  Asynchronous on stream.
 */
int msa_fwd(const msa_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
            const int32_t* sel, uint16_t* o, float* lse, int32_t* d_status, void* ws,
            size_t ws_bytes, void* stream);

/* Block scorer and top-k selection: writes the sel array that msa_build_k2q
 * and msa_fwd consume ("msa_bindings" page, MSAKernels.fmha_sm100, the scorer
 * launcher; "msa_schedule" page, INDEX_DIM = 128 index dims per index head).
 * The pages name the scorer but not its score; this call computes:
 *  - per index head, the pooled index query of every query chunk and the
 *    pooled index key of every key block: the mean of the tokens' index
 *    vectors inside the document (fp32 sum in token order, divided by the
 *    token count, rounded to bf16);
 *  - score(chunk, block) = the fp32 dot product of the two pooled vectors,
 *    summed in ascending index-dim order;
 *  - sel[hi][g] = the chunk's diagonal block (the one holding its first
 *    query), then the topk - 1 blocks before it with the highest scores (a tie
 *    goes to the lower block) by descending score, then -1; every entry is a
 *    document-local block id and causal, so the result is a valid selection.
 * q_index, k_index  device bf16 [T, Hi, 128]: index query / key of each token
 *                   (compact token rows, the cu_seqlens order).
 * sel               device int32 [Hi, NC, topk] out.
 * ws                device workspace of at least msa_workspace_bytes() bytes
 *                   (it holds the pooled vectors).
 * Deterministic: the same inputs give the same sel on every run.  Returns
 * MSA_ERR_INVALID_ARGUMENT for a null or misaligned pointer or a short ws;
 * device-detected document errors go to *d_status.  Asynchronous on stream. */
int msa_select_topk(const msa_problem* p, const uint16_t* q_index, const uint16_t* k_index, int32_t* sel,
                    int32_t* d_status, void* ws, size_t ws_bytes, void* stream);

/* Forward work plan ("msa_bindings" page, MSAKernels.fmha_sm100_plan, the
 * planner launcher; "msa_schedule" page, MSABackwardSchedule's
 * scheduler_metadata and work_count): the forward's work items, built on the
 * device with no host synchronisation.
 * One item per (index head, query chunk), written as a scheduler_metadata row
 * in the pages' column order (MSA_TASK_META_COLS): index_head, row_linear =
 * the global query chunk, q_begin = its first token row, q_count = its token
 * count, document_ordinal, document_local_kblock = the key block holding its
 * first query.  Rows are ordered longest first: descending number of selected
 * blocks, ties in (index head, chunk) order, items selecting no block last, so
 * a persistent walk over them meets the long items first.
 * sel                 device int32 [Hi, NC, K], as for msa_fwd.
 * scheduler_metadata  device int32 [Hi * NC, 6] out: every item, once.
 * work_count          device int32 [1] out: items that select at least one
 *                     block (the rows before the empty ones).
 * ws                  workspace of at least msa_workspace_bytes() bytes.
 * Deterministic.  Asynchronous on stream; argument errors are return codes,
 * document errors go to *d_status. */
int msa_plan_forward(const msa_problem* p, const int32_t* sel, int32_t* scheduler_metadata,
                     int32_t* work_count, int32_t* d_status, void* ws, size_t ws_bytes, void* stream);

/* msa_fwd walking the items in the order of a plan written by
 * msa_plan_forward for the same problem and selection (the w-th item the
 * persistent CTAs take is row w of scheduler_metadata).  O and LSE are the
 * same, bit for bit, as msa_fwd's: every item is computed the same way
 * whichever CTA takes it. */
int msa_fwd_planned(const msa_problem* p, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                    const int32_t* sel, const int32_t* scheduler_metadata, uint16_t* o, float* lse,
                    int32_t* d_status, void* ws, size_t ws_bytes, void* stream);

/* -------------------------------------------------------------------------
 * Serving: a paged key/value cache in 4 bits and the operators over it.
 *
 * The pages describe the training pass only; these calls have no counterpart
 * there.  They carry the same method to a serving step: a batch of requests,
 * each with `past` cached tokens and some new ones, whose new tokens attend
 * the top-k selected key blocks of their own request.  One step is
 *   msa_cache_step    block table, slots and query chunks from the lengths,
 *   msa_cache_append  the new tokens' K, V and index keys into the cache,
 *   msa_cache_select  the key blocks of every query chunk,
 *   msa_cache_fwd     attention over the selected blocks,
 * each asynchronous on its stream, with fixed buffers and no workspace, so a
 * step can be captured into a CUDA graph and replayed.  The step's tables are
 * read on the device only: no call needs a length on the host.
 *
 * Errors.  A call that finds *d_status set does nothing.  A call other than
 * msa_cache_step that sets it itself leaves out what is at fault and, besides,
 * whatever parts of its own launch come up behind the error: which these are is
 * not determined (a row of a tensor, a head of it or 16 of its dims may be left
 * as it was).  What it does write is what it would have written without the
 * error, but for selections over a bad page.
 *
 * A page holds one key block of one cache (block_size tokens of every KV
 * head).  Position p of request r lives in page block_table[r][p / B], at
 * offset p % B; its slot is page * B + offset.  The new tokens of a request
 * are cut into query chunks: tokens of equal position / 8, as in the training
 * pass, so a chunk lies in one page.
 *
 * Cache layout, uint8 [num_pages, Hkv, B / 64, MSA_CACHE_TILE_BYTES]: per page
 * and head, tiles of 64 tokens, each
 *   K codes  [64 tokens][64 bytes]     at 0
 *   K scales [64 tokens][8]            at 4096
 *   V codes  [64 tokens][64 bytes]     at 4608, byte o of the plane stored at
 *                                      o ^ ((token & 12) << 3)
 *   V scales [8][64 tokens]            at 8704
 * Byte i of a token's codes holds dims 2i (low half) and 2i + 1 (high half)
 * as e2m1 (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
 * 4, 6; a zero is written without a sign); scale j is the e4m3 scale of dims 16j .. 16j + 15.  A K value is
 * code * scale * 2^k_exp, a V value code * scale * 2^v_exp; without the
 * power of two it is exact in fp16 and bf16.
 * ------------------------------------------------------------------------- */

/* num_requests   R, rows of the block table (batch slots), 1 .. 8192.
 * num_pages      P, pages of the cache, 1 .. 2^24.
 * max_blocks     M, block-table columns, 1 .. 49152; M * B tokens at most.
 * num_q_heads    Hq = 16 * num_kv_heads; index heads = KV heads (<= 1024).
 * head_dim 128.  block_size B: 64 or 128.  query_chunk 8.  topk 1 .. 32.
 * token_cap      T, rows of the step's token tensors (new tokens fit in it;
 *                rows behind the last new token are padding), 1 .. 2^24.
 * chunk_cap      NC, rows of the step's chunk table, 1 .. 2^24.
 * k_exp, v_exp   exponents of the cache's values, -32 .. 32: an e4m3 scale
 *                spans 2^-9 .. 448, so groups whose largest element is below
 *                0.09 * 2^exp lose precision and those above 2688 * 2^exp
 *                saturate.  The same values in every call on one cache.
 * softmax_scale  scale applied to q.k, > 0 and finite. */
typedef struct {
  int32_t num_requests;
  int32_t num_pages;
  int32_t max_blocks;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t query_chunk;
  int32_t topk;
  int32_t token_cap;
  int32_t chunk_cap;
  int32_t k_exp;
  int32_t v_exp;
  float softmax_scale;
} msa_cache_problem;

enum { MSA_CACHE_TILE_BYTES = 9216 };
/* Columns of a row of the step's chunk table: request, first token row, token
 * count (1 .. 8), position of the first token.  A row with request -1 is
 * padding. */
enum { MSA_CHUNK_COLS = 4 };

/* Bytes of the cache of p (0 if p is invalid). */
size_t msa_cache_bytes(const msa_cache_problem* p);
/* Rows of the chunk table that hold every chunk of any `tokens` new tokens of
 * num_requests requests: min(tokens, tokens / 8 + 2 * num_requests). */
int64_t msa_cache_chunk_bound(int64_t tokens, int64_t num_requests);

/* Block table, slot map, positions and query chunks of one step, from the
 * lengths on the device.
 * new_lens      device int32 [R]: new tokens of each request, 0 for an idle
 *               one, -1 for one that has finished and gives its pages back.
 * seq_lens      device int32 [R]: cached tokens before the step.
 * ring          device int32 [2]: first entry and count of the free pages in
 *               free_ring.
 * free_ring     device int32 [P] in/out: page ids in a ring.  New blocks take
 *               pages from its front in (request, block) order; pages given
 *               back join its end in the same order and are not handed out
 *               in the same step.
 * block_table   device int32 [R, M] in/out: only the entries of the step's
 *               new blocks are written.
 * seq_lens_out  device int32 [R] out: past + new, 0 for a finished request.
 * ring_out      device int32 [2] out.  seq_lens_out and ring_out may be
 *               seq_lens and ring themselves.
 * cu_tokens     device int32 [R + 1] out: first token row of each request.
 * slot_map      device int64 [T] out: slot of each new token, -1 for padding.
 * positions     device int32 [T] out: its position, -1 for padding.
 * chunks        device int32 [NC, 4] out (MSA_CHUNK_COLS), in token order,
 *               -1 in every column of padding.
 * *d_status: MSA_ERR_CAPACITY when the new tokens, their chunks, a request's
 * blocks or the pages needed exceed T, NC, M or the free pages;
 * MSA_ERR_INVALID_CACHE when a length or the ring is out of range.  Nothing
 * is written then.  Deterministic. */
int msa_cache_step(const msa_cache_problem* p, const int32_t* new_lens, const int32_t* seq_lens,
                   const int32_t* ring, int32_t* free_ring, int32_t* block_table, int32_t* seq_lens_out,
                   int32_t* ring_out, int32_t* cu_tokens, int64_t* slot_map, int32_t* positions,
                   int32_t* chunks, int32_t* d_status, void* stream);

/* Rounds K and V of the new tokens to 4 bits and writes them to their slots,
 * and keeps the pooled index keys that msa_cache_select scores.
 * Rounding, per token, head and 16 dims: scale = e4m3(max |x| * 2^-exp / 6),
 * to nearest even, at most 448; code = e2m1(x * 2^-exp / scale), to nearest
 * even, at most 6; a zero scale gives zeros.  A group that holds an infinity
 * or a NaN reads back as NaN.
 * k, v         device bf16 [T, Hkv, 128].
 * slot_map     device int64 [T]; -1 leaves the row out.  A slot outside the
 *              cache is left out and sets MSA_ERR_INVALID_CACHE.  A slot that
 *              appears twice holds one of its rows, in part perhaps each.
 * cache        device uint8, msa_cache_bytes(p).
 * k_index      device bf16 [T, Hkv, 128], index key of each new token, or
 *              NULL: cu_tokens, chunks, index_tail and index_pool are then
 *              not used and may be NULL.
 * cu_tokens, chunks  as msa_cache_step wrote them.  A chunk row that does not
 *              fit (the token rows, its block, max_blocks) is left out and
 *              sets MSA_ERR_INVALID_CACHE.
 * index_tail   device bf16 [R, 2, B, Hkv, 128] in/out: index keys of each
 *              request's incomplete block b, at [r][b & 1][position % B].  (The
 *              rows that a request's first block is completed with are still
 *              there after the call, unless the call's last block of the
 *              request is an even number of blocks, and not 0, behind it.)
 * index_pool   device bf16 [P, Hkv, 128] out: for each block that this call
 *              completes, the mean of its tokens' index keys (fp32 sum in
 *              token order, divided by B, rounded to bf16). */
int msa_cache_append(const msa_cache_problem* p, const uint16_t* k, const uint16_t* v,
                     const uint16_t* k_index, const int64_t* slot_map, const int32_t* cu_tokens,
                     const int32_t* chunks, uint8_t* cache, uint16_t* index_tail, uint16_t* index_pool,
                     int32_t* d_status, void* stream);

/* The values that the cache holds, rounded to bf16 (exact but for results
 * outside bf16's normal range): for a prefill over cached tokens, to move a
 * request, or to look at the cache.
 * slots  device int64 [T] (any slots, in any order); -1 leaves the row of k
 *        and v as it was, a slot outside the cache does so too and sets
 *        MSA_ERR_INVALID_CACHE.
 * k, v   device bf16 [T, Hkv, 128] out. */
int msa_cache_read(const msa_cache_problem* p, const int64_t* slots, const uint8_t* cache, uint16_t* k,
                   uint16_t* v, int32_t* d_status, void* stream);

/* Top-k key blocks of every query chunk of a step, by the rule of
 * msa_select_topk: the chunk's index query is the mean of its new tokens'
 * index queries, a block's key its row of index_pool, the score their fp32
 * dot product summed in ascending dim order; the block that holds the chunk
 * first, then the topk - 1 earlier ones with the highest scores (a tie goes
 * to the lower block) by descending score, then -1.
 * q_index      device bf16 [T, Hkv, 128].
 * index_pool   device bf16 [P, Hkv, 128]: every block before a chunk's own is
 *              complete, so its row is there.
 * block_table, chunks  as msa_cache_step wrote them.
 * sel          device int32 [Hkv, NC, topk] out; rows of padding chunks are
 *              left as they were.
 * A chunk row that does not fit and a page outside the cache set
 * MSA_ERR_INVALID_CACHE: such a chunk's rows are left as they were, and the
 * rows of the page's request mean nothing.
 * Deterministic where no error is found; a NaN score may take any rank, the
 * selection stays valid. */
int msa_cache_select(const msa_cache_problem* p, const uint16_t* q_index, const uint16_t* index_pool,
                     const int32_t* block_table, const int32_t* chunks, int32_t* sel, int32_t* d_status,
                     void* stream);

/* Attention of the new tokens over the selected blocks of the cache: for each
 * query row, softmax(scale * q k^T) over the keys of its chunk's selected
 * blocks at or before its own position, times V.  The new tokens' own keys
 * must be in the cache (msa_cache_append first).
 * q            device bf16 [T, Hq, 128].
 * sel          device int32 [Hkv, NC, topk]: blocks of the chunk's request,
 *              negative for an empty slot; distinct, and none behind the
 *              chunk's own block (MSA_ERR_INVALID_SELECTION otherwise, and
 *              the chunk's rows of that head are left as they were).
 * o            device bf16 [T, Hq, 128] out;  lse device fp32 [T, Hq] out
 *              (natural log).  A row that attends no key has o = 0 and lse =
 *              -inf.  Rows that no chunk covers are left as they were.
 * Cache bytes of keys that no query may attend may hold anything.
 * Deterministic where no error is found. */
int msa_cache_fwd(const msa_cache_problem* p, const uint16_t* q, const uint8_t* cache,
                  const int32_t* block_table, const int32_t* chunks, const int32_t* sel, uint16_t* o,
                  float* lse, int32_t* d_status, void* stream);

/* -------------------------------------------------------------------------
 * Norm and rotary positions of queries, keys and index vectors: what lies
 * between the projections and msa_select_topk / msa_fwd / msa_cache_append, and
 * its gradients behind msa_bwd.  (The pages start from tensors that have both;
 * these calls have no counterpart there.)
 *
 * Every head (128 dims) of every token of a tensor is normed (MSA_ROPE_NORM),
 *   n = x * (w + weight_offset) / sqrt(mean(x^2) + eps),
 * and its first R = rotary_dim dims are rotated (MSA_ROPE_ROTATE): pair p of
 * R / 2 is dims (p, p + R / 2), or (2p, 2p + 1) where `adjacent` is set, and
 *   (a, b) -> cos_scale * (a cos t - b sin t, b cos t + a sin t)
 * with t = 2 pi * turns[p] / 2^64 * position[axis[p]]: each pair follows one of a
 * token's num_axes positions (one for text; time, height and width of images and
 * video).  Angles are formed in 64-bit fixed point, which loses nothing at any
 * position; the table's own rounding, 2^-65 of a turn, counts once a position: 2^-34
 * at position 2^31, less than fp32 tells.  All else is fp32, rounded to bf16 once.
 * Rows may hold any finite values.  Weights (offset added) times cos_scale may reach
 * 2^62, and their products with the gradients 2^100: beyond, fp32 may overflow.
 *
 * The tensors of one call share a launch and their tokens' angles.  x and y may
 * be strided (parts of one projection's output), with strides in elements.
 * ------------------------------------------------------------------------- */
enum { MSA_ROPE_Q = 0, MSA_ROPE_K = 1, MSA_ROPE_Q_INDEX = 2, MSA_ROPE_K_INDEX = 3, MSA_ROPE_V = 4, MSA_ROPE_TENSORS = 5 };
enum { MSA_ROPE_NORM = 1, MSA_ROPE_ROTATE = 2, MSA_ROPE_PER_HEAD = 4, MSA_ROPE_WEIGHT_FP32 = 8 };

/* heads     of this tensor; 0: the call has no such tensor.
 * flags     MSA_ROPE_NORM, MSA_ROPE_ROTATE; MSA_ROPE_PER_HEAD: a weight per head
 *           ([heads, 128], else [128]); MSA_ROPE_WEIGHT_FP32: the weight (and
 *           its gradient) is fp32, else bf16.
 * weight    device, or NULL for a norm without one (w + weight_offset is then 1).
 * x_token, x_head, y_token, y_head  elements from one token's row, and one head's,
 *           to the next: multiples of 8 from 128 to 2^38 that keep the rows apart. */
typedef struct {
  int32_t heads;
  uint32_t flags;
  const void* weight;
  int64_t x_token, x_head, y_token, y_head;
} msa_rope_tensor;

/* One pair: turns per position in units of 2^-64, and the position's column. */
typedef struct {
  uint64_t turns;
  int32_t axis;
  int32_t reserved;
} msa_rope_pair;

/* tokens        rows of every tensor, 0 .. 2^24.
 * head_dim      128.
 * rotary_dim    R: 32, 64, 96 or 128 (0 if no tensor is rotated).
 * num_axes      columns of the positions, 1 .. 4.
 * eps           2^-100 .. 2^100.
 * cos_scale     > 0 and finite; 1 but for stretched contexts.
 * pairs         device [R / 2], written from msa_rope_pairs' output.  An axis out
 *               of range counts as 0 and sets MSA_ERR_INVALID_ARGUMENT; parts of
 *               the call that come up behind that are left out.
 * zero_padding  what becomes of the output rows (y, dx) of tokens that are padding:
 *               0: they are left as they were, 1: they are zeros (outputs in new
 *               memory, gradients that a sum over all rows follows). */
typedef struct {
  int32_t tokens;
  int32_t head_dim;
  int32_t rotary_dim;
  int32_t num_axes;
  int32_t adjacent;
  float eps;
  float weight_offset;
  float cos_scale;
  const msa_rope_pair* pairs;
  msa_rope_tensor tensor[MSA_ROPE_TENSORS];
  int32_t zero_padding;
} msa_rope_problem;

/* Fills pairs[0 .. num_pairs) on the host from angular frequencies (radians per
 * position, as rotary tables give them) and position columns (NULL: 0).  turns is
 * the frequency's quotient by 2 pi, modulo 1, rounded once to 2^-64 (frequencies of
 * up to 2^38; beyond, within 2^-100 of the quotient). */
int msa_rope_pairs(const double* inv_freq, const int32_t* axes, int32_t num_pairs, msa_rope_pair* pairs);

/* The forward.
 * x, y       host arrays of four device pointers (MSA_ROPE_Q .. MSA_ROPE_K_INDEX; p's
 *            V tensor is not used): bf16 rows in and out.  Entries of tensors with
 *            no heads are not looked at.  y may be x itself, with the same strides;
 *            what is written shares no memory with other tensors of a call, here
 *            and below, but where it is said.
 * positions  device int32 [tokens, num_axes].  A token whose first position is
 *            negative is padding: its rows of y are left as they were, or zeros
 *            (zero_padding).  Other columns may be negative.
 * Deterministic; a row's result does not depend on the call's other rows. */
int msa_norm_rope(const msa_rope_problem* p, const uint16_t* const* x, const int32_t* positions, uint16_t* const* y,
                  int32_t* d_status, void* stream);

/* Bytes of workspace of msa_norm_rope_bwd (0 if p is invalid; at least 256). */
size_t msa_norm_rope_bwd_bytes(const msa_rope_problem* p);

/* Its gradients.
 * dy         bf16, laid out by p's y strides: the gradients of y.
 * x          the forward's input (not its output: with y = x it is gone).
 * dx         bf16 out, laid out by p's x strides; may be x itself, or dy itself
 *            where the strides agree.  Rows of padding are left as they were, or
 *            zeros (zero_padding).
 * dw         host array of four device pointers, entries NULL where the gradient
 *            is not wanted or there is no weight: [128] or [heads, 128], in the
 *            weight's type, summed in fp32 over the tokens that are no padding
 *            (and over the heads that share it).  Overwritten, not added to.  The
 *            chains of additions grow with the rows: 131072 tokens x 152 heads make
 *            2,185 long ones, and sums that are off by 0.2 x 2^-24 of the sum of the
 *            magnitudes, 7.3 x 2^-24 where all products have one sign.
 * ws         msa_norm_rope_bwd_bytes(p), overwritten before it is read.
 * Deterministic. */
int msa_norm_rope_bwd(const msa_rope_problem* p, const uint16_t* const* dy, const uint16_t* const* x,
                      const int32_t* positions, uint16_t* const* dx, void* const* dw, int32_t* d_status, void* ws,
                      size_t ws_bytes, void* stream);

/* msa_cache_append of tensors that are not normed and rotated yet, with all that
 * a step's other calls need, in one launch:
 *  - q and q_index normed and rotated to q_out and q_index_out, as msa_norm_rope
 *    does;
 *  - K normed, rotated and rounded to 4 bits by msa_cache_append's rule, V rounded
 *    as it is, both written to the tokens' slots.  K is not rounded to bf16 in
 *    between: its codes and scales are those of the exact value of y (what lies
 *    closer to a border than fp32 can tell is computed again in pairs of fp32, within
 *    2^-38, which leaves about one value in 10^10).  A value beyond fp32's range
 *    makes its group NaN, as an infinite one does;
 *  - index keys normed, rotated and rounded to bf16 as msa_norm_rope does, and kept
 *    by msa_cache_append's rule (index_tail and index_pool hold the same, bit for
 *    bit, as after the two calls).
 * p          the tensors of the step: K and V with c's num_kv_heads and V without
 *            flags; Q with c's num_q_heads or 0 heads (q and q_out are not used
 *            then); Q_INDEX with num_kv_heads or 0; K_INDEX with num_kv_heads, or
 *            0 in a call without index keys (its other arguments may be NULL).
 *            K and V are written to the cache: their y strides, and K_INDEX's, are
 *            not used.  p.tokens = c.token_cap.
 * positions  device int32 [T, num_axes]; msa_cache_step's positions where there is
 *            one axis.  A token whose first position is negative is padding: none of
 *            its rows are written (but zeros to q_out and q_index_out, with
 *            zero_padding).  A token whose slot is -1 leaves out K and V.  A
 *            slot outside the cache, or one beside a negative first position, leaves
 *            them out too and sets MSA_ERR_INVALID_CACHE.  With index keys, the rows
 *            that chunks covers must not be padding.
 * Other arguments as for msa_cache_append.  Deterministic where no error is found. */
int msa_cache_append_rope(const msa_cache_problem* c, const msa_rope_problem* p, const uint16_t* q, const uint16_t* k,
                          const uint16_t* v, const uint16_t* q_index, const uint16_t* k_index,
                          const int32_t* positions, const int64_t* slot_map, const int32_t* cu_tokens,
                          const int32_t* chunks, uint16_t* q_out, uint16_t* q_index_out, uint8_t* cache,
                          uint16_t* index_tail, uint16_t* index_pool, int32_t* d_status, void* stream);

/* Self-test of the bounded device waits (no counterpart in the pages).
 * Launches one small kernel that waits, with the same bounded mbarrier wait
 * every kernel of this library uses, for an mbarrier phase that nothing
 * completes.  After the wait limit (2 s) the kernel writes MSA_ERR_TIMEOUT to
 * *d_status (first error wins) and returns normally: no fault, no hang, and
 * the CUDA context stays usable.  d_status: device int32, caller-owned.
 * Returns MSA_ERR_INVALID_ARGUMENT for a null or misaligned d_status,
 * MSA_ERR_CUDA if the launch fails.  Asynchronous on stream. */
int msa_selftest_wait_timeout(int32_t* d_status, void* stream);

/* Host-side walk rule ("msa_schedule" page): rows_per_cta, chunk_map and
 * grid_launch_bound.  chunk_map writes (full, tail, grid) to out3. */
int32_t msa_rows_per_cta(int64_t num_rows);
void msa_chunk_map(int64_t num_rows, int32_t rows_per_cta, int32_t num_sms, int64_t* out3);
int64_t msa_grid_launch_bound(int64_t capacity, int32_t num_sms);

/* Memoised device queries ("kernels" page, sm_capability and sm_count: a
 * device's capability cannot change, so it is looked up once per device). */
int msa_device_capability(int32_t device, int32_t* major, int32_t* minor);
int msa_device_sm_count(int32_t device, int32_t* sm_count);

/* Static text for a status code. */
const char* msa_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MSA_H_ */
