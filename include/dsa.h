/*
 * dsa.h -- C ABI of the DSA sparse-attention hot path on GB300 (sm_103a).
 *
 * The path has three stages over a block-paged KV cache:
 *   1. indexer score  -- "Day-0 Adaptation of Trillion-Parameter MoE Models on
 *      Domestic GPUs", section 3 (1) Index Selection: a lightweight similarity
 *      score of every cached position against the query;
 *   2. top-K          -- same passage (the K best positions found block by
 *      block, then combined across blocks), with the deterministic tie rule of
 *      "Day-0 Adaptation of Ultra-Large-Scale MoE Models on Heterogeneous AI
 *      Accelerators", section 4 (equal scores: the lower position wins);
 *   3. sparse attention -- first page, section 3 (3): exact softmax attention
 *      over the selected positions only, with separate decode (memory-bound)
 *      and prefill (compute-bound) paths.
 * The cache layout follows first page, section 3 (2): pages of `block_size`
 * consecutive positions stored contiguously, an index table jumping between
 * pages.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every tensor pointer is a DEVICE pointer owned by the caller; the library
 *    never allocates, frees or keeps a pointer after a call returns.
 *  - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream) and launches kernels only: no host synchronisation, no
 *    allocation, so the calls may be captured into a CUDA graph.
 *  - Tensors are dense and row-major in the shapes written next to them, except
 *    the KV pools, whose rows are `*_row_stride` elements apart.
 *  - Return value: DSA_OK, or a negative DSA_ERR_* code for errors the host can
 *    see (bad pointer, shape, dtype or workspace).  Then nothing was launched
 *    and the message is in dsa_last_error_string().
 *  - Errors that depend on device data (a block-table entry outside
 *    [0, num_blocks), an index past its sequence, a bounded wait that ran out)
 *    never trap: the offending position or row is skipped (score -inf, row left
 *    out of the softmax) and a DSA_STATUS_* bit is OR-ed into the status word
 *    at the start of the call's workspace; dsa_get_status() reads it.
 *  - Workspaces: query the size with the matching dsa_*_workspace_size(), pass a
 *    caller-owned device buffer of at least that size, 256-byte aligned and
 *    ZERO-FILLED before its first use.  The library leaves it in a reusable
 *    state after every call (counters return to zero; the status word is sticky
 *    until read with clear=1).  A workspace may serve different calls in turn;
 *    calls that share one must not overlap on the GPU (issue them on one
 *    stream, or order the streams).
 */
#ifndef DSA_H_
#define DSA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* dsa_stream_t; /* = cudaStream_t */

/* host-visible return codes */
#define DSA_OK 0
#define DSA_ERR_INVALID (-1)     /* null pointer, bad shape, K, stride or layout */
#define DSA_ERR_UNSUPPORTED (-2) /* no kernel for this dtype / head count / dims */
#define DSA_ERR_WORKSPACE (-3)   /* workspace missing, misaligned or too small */
#define DSA_ERR_CUDA (-4)        /* a CUDA call failed; see dsa_last_error_string() */
#define DSA_ERR_TIMEOUT (-5)     /* reported by dsa_get_status() users, see below */

/* device status bits (dsa_get_status) */
#define DSA_STATUS_BAD_BLOCK 0x1  /* block-table entry outside [0, num_blocks) */
#define DSA_STATUS_BAD_INDEX 0x2  /* selected index >= its sequence length */
#define DSA_STATUS_BAD_LENGTH 0x4 /* seq_len > max_blocks_per_seq*block_size, or > ld */
#define DSA_STATUS_TIMEOUT 0x8    /* a bounded device wait gave up */

/* element types */
#define DSA_BF16 0     /* bfloat16 */
#define DSA_FP8_E4M3 1 /* OCP FP8 E4M3 ("fn": no infinities) */

/*
 * Paged cache layout ("Day-0 Adaptation of Trillion-Parameter MoE Models on
 * Domestic GPUs", section 3 (2)).  Logical position p of sequence b is stored
 * in physical row  block_table[b][p / block_size] * block_size + p % block_size
 * of every pool (KV pool, indexer-key pool).  Unused table entries may hold
 * any value; they are never read.
 */
typedef struct dsa_paged_layout {
  int32_t block_size;          /* positions per page, 1..1024 (64 in the workloads) */
  int32_t num_blocks;          /* pages in each pool (NB) */
  int32_t max_blocks_per_seq;  /* row length of block_table */
  int32_t batch;               /* number of sequences B */
  int32_t max_seq_len;         /* host-known bound: every seq_lens[b] <= max_seq_len */
  int32_t reserved_;           /* set to 0 */
  const int32_t* block_table;  /* device [batch][max_blocks_per_seq] */
  const int32_t* seq_lens;     /* device [batch]: cached positions L_b (query included) */
} dsa_paged_layout;

/* ---------------------------------------------------------------------------
 * Stage 1: indexer score.
 * Source: "Day-0 Adaptation of Trillion-Parameter MoE Models on Domestic GPUs",
 * section 3 (1) (each cached position scored by its similarity to the
 * query through low-dimensional keys), read as
 *     scores[r][p] = sum_h w[r][h] * max(0, sum_d q_idx[r][h][d] * k_idx[p][d])
 * for every position p the query may see: p <= q_pos[r] and p < L_b (causal,
 * the current position included).  Entries of the row past the last eligible
 * position are not part of the result and may be left untouched.
 * Accumulation is fp32; with integer-valued q_idx/k_idx/w
 * (the pages' workloads) the scores are exact integers below 2^24.
 *
 *  layout      paged layout; only block_table/seq_lens rows of the queried
 *              sequences are read
 *  q_idx       [Nq][H_i][D_i] of `dtype` -- indexer queries
 *  w           [Nq][H_i] fp32 -- head weights
 *  kidx_pool   [num_blocks][block_size][D_i] of `dtype` -- indexer keys
 *  dtype       DSA_BF16 or DSA_FP8_E4M3 (q_idx and kidx_pool share it)
 *  H_i, D_i    indexer heads (1..128) and dim (32, 64 or 128)
 *  q_seq       [Nq] sequence of each query, or NULL: query r is sequence r
 *  q_pos       [Nq] absolute position of each query, or NULL: L_b - 1 (decode)
 *  scores      [Nq][ld] fp32 output; ld >= eligible positions of every row
 *  ws          workspace of dsa_index_score_workspace_size() bytes
 * Errors: DSA_ERR_INVALID for null pointers, Nq < 0, ld < 1 or a bad layout;
 * DSA_ERR_UNSUPPORTED for other H_i/D_i/dtype and for Nq > 65535 (call in
 * chunks of queries).  Device: out-of-range block ids give -inf scores and
 * DSA_STATUS_BAD_BLOCK.
 */
size_t dsa_index_score_workspace_size(int Nq, int H_i, int D_i, int64_t ld);
int dsa_index_score(const dsa_paged_layout* layout, const void* q_idx, const float* w,
                    const void* kidx_pool, int dtype, int H_i, int D_i,
                    const int32_t* q_seq, const int32_t* q_pos, int Nq, float* scores,
                    int64_t ld, void* ws, size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Stage 1, prefill form: all Nq queries belong to sequence `seq` and query r
 * sits at position q_pos[r] (q_pos NULL: position r).  Same scores as
 * dsa_index_score with q_seq[r] = seq.  Source: "Day-0 Adaptation of
 * Trillion-Parameter MoE Models on Domestic GPUs", section 3 (3): the prefill
 * stage processes the whole prompt at once and is compute-intensive, so the
 * queries share every key tile (a dense causal contraction on tensor cores).
 * Errors as for dsa_index_score; seq must be in [0, batch).
 */
size_t dsa_index_score_prefill_workspace_size(int Nq, int H_i, int D_i, int64_t ld);
int dsa_index_score_prefill(const dsa_paged_layout* layout, int seq, const void* q_idx,
                            const float* w, const void* kidx_pool, int dtype, int H_i, int D_i,
                            const int32_t* q_pos, int Nq, float* scores, int64_t ld, void* ws,
                            size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Stage 2: top-K selection.
 * Source: "Day-0 Adaptation of Trillion-Parameter MoE Models on Domestic GPUs",
 * section 3 (1) (selection done per block of positions and then combined
 * over the blocks, with no sort of the whole row); tie rule from "Day-0
 * Adaptation of Ultra-Large-Scale MoE Models on Heterogeneous AI
 * Accelerators", section 4: among equal scores the lower position wins.
 * For row r, among positions 0..n_eligible[r]-1, keep the min(K, n) positions
 * with the largest score (scores compared as values: -0.0 ties +0.0), write
 * them to idx[r] in ascending position order and pad with -1.
 *
 *  scores      [Nq][ld] fp32 (finite or -inf; NaN ranks below every value)
 *  n_eligible  [Nq] int32, each in [0, ld] (larger values are clamped to ld
 *              and flagged DSA_STATUS_BAD_LENGTH)
 *  K           1..65536
 *  idx         [Nq][K] int32 output
 *  ws          workspace of dsa_topk_workspace_size() bytes
 */
size_t dsa_topk_workspace_size(int Nq, int64_t ld, int K);
int dsa_topk(const float* scores, int64_t ld, const int32_t* n_eligible, int Nq, int K,
             int32_t* idx, void* ws, size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * dsa_topk_noalloc: the selection of dsa_topk (same arguments and results,
 * minus the workspace) for callers that cannot allocate device memory: code
 * given a stream but no allocator by the framework that owns the GPU's
 * memory, real-time threads that must not wait on allocator locks, and
 * deployments whose device memory is fully divided up in advance.  The pages
 * have no counterpart; this is a deployment convenience.
 *  Scratch: one fixed array of DSA_TOPK_NOALLOC_SCRATCH_BYTES inside the
 *    library, present on every GPU that loads it until the process exits.  No
 *    call allocates or frees device memory.
 *  First call on a device: looks up the array's device address (once per
 *    device, with that device current) and keeps it for the life of the
 *    process.  Make that first call before any stream capture.  A
 *    cudaDeviceReset() of that device invalidates the kept address: do not
 *    reset a device between calls of this function in one process.
 *  Limit: a problem whose scratch would exceed the array
 *    (dsa_topk_workspace_size() > DSA_TOPK_NOALLOC_SCRATCH_BYTES) is rejected
 *    with DSA_ERR_WORKSPACE and a message; nothing is launched.
 *  Sharing: every call uses the same array.  Calls that overlap on the GPU
 *    (unordered streams, several host threads) race and corrupt each other's
 *    results; order them on one stream.  The status word is cleared at the
 *    start of each call and cannot be read back.
 */
#define DSA_TOPK_NOALLOC_SCRATCH_BYTES (8u << 20)
int dsa_topk_noalloc(const float* scores, int64_t ld, const int32_t* n_eligible, int Nq, int K,
                     int32_t* idx, dsa_stream_t stream);
/* The size of that fixed array as this build of the library has it
 * (DSA_TOPK_NOALLOC_SCRATCH_BYTES), for callers that load the library at run
 * time and cannot see the header's define. */
size_t dsa_topk_noalloc_scratch_bytes(void);

/* ---------------------------------------------------------------------------
 * Stage 3a: sparse attention, decode (one query per sequence).
 * Source: "Day-0 Adaptation of Trillion-Parameter MoE Models on Domestic GPUs",
 * section 3 (3) (decode: one token per step, memory-bandwidth-bound) and the
 * execution chain of "Day-0 Adaptation of Ultra-Large-Scale MoE Models on
 * Heterogeneous AI Accelerators", section 4 (cache gather + sparse attention).
 * For sequence b and head h, over the selected positions j (idx[b][*] >= 0),
 * whose rows are gathered through the block table:
 *     z_j = sm_scale * q[b][h] . K_j,   out[b][h] = sum_j softmax(z)_j V_j,
 *     lse[b][h] = log sum_j exp(z_j)
 * One shared K/V head (multi-query); fp32 accumulation and softmax.
 *
 *  q            [B][Hq][Dqk] bf16
 *  k_pool       physical rows of Dqk bf16, k_row_stride elements apart
 *  v_pool       physical rows of Dv bf16, v_row_stride elements apart; may be
 *               k_pool itself (latent cache: V = first Dv dims of the K row)
 *  Hq           1..64 query heads; Dqk, Dv multiples of 8 (>= 8), Dv <= 512,
 *               Hq * Dqk * 2 + 4 * (Dqk + Dv) <= 200 KB (q of one query held in
 *               shared memory); B (Nq for prefill) <= 65535.  Other shapes
 *               return DSA_ERR_UNSUPPORTED.
 *  idx          [B][K] int32 positions from dsa_topk (-1 = padding, skipped)
 *  out          [B][Hq][Dv] bf16 output (0 for a row with no selected position)
 *  lse          [B][Hq] fp32 output, or NULL (-inf for an empty row)
 *  ws           workspace of dsa_sparse_attn_decode_workspace_size() bytes
 * Device errors: an index >= L_b or a bad block id skips that row and sets
 * DSA_STATUS_BAD_INDEX / DSA_STATUS_BAD_BLOCK.
 */
size_t dsa_sparse_attn_decode_workspace_size(int B, int Hq, int Dqk, int Dv, int K);
int dsa_sparse_attn_decode(const dsa_paged_layout* layout, const void* q, const void* k_pool,
                           int64_t k_row_stride, const void* v_pool, int64_t v_row_stride,
                           int Hq, int Dqk, int Dv, const int32_t* idx, int K, float sm_scale,
                           void* out, float* lse, void* ws, size_t ws_bytes,
                           dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Stage 3b: sparse attention, prefill (many queries, each with its own
 * selected set).  Source: "Day-0 Adaptation of Trillion-Parameter MoE Models
 * on Domestic GPUs", section 3 (3) (prefill: whole prompt at once,
 * compute-intensive).  Same arithmetic as stage 3a for each query r of
 * sequence q_seq[r]:
 *  q            [Nq][Hq][Dqk] bf16
 *  q_seq        [Nq] int32 sequence of each query, or NULL: all in sequence 0
 *  q_pos        [Nq] int32 absolute position of each query, or NULL.  When
 *               given, only the first min(K, q_pos+1) entries of idx[r] are
 *               read and an index > q_pos (non-causal) is skipped and flagged
 *               DSA_STATUS_BAD_INDEX
 *  idx          [Nq][K] int32
 *  out          [Nq][Hq][Dv] bf16, lse [Nq][Hq] fp32 or NULL
 *  ws           workspace of dsa_sparse_attn_prefill_workspace_size() bytes
 * Other arguments and errors as for stage 3a.
 */
size_t dsa_sparse_attn_prefill_workspace_size(int Nq, int Hq, int Dqk, int Dv, int K);
int dsa_sparse_attn_prefill(const dsa_paged_layout* layout, const void* q, const void* k_pool,
                            int64_t k_row_stride, const void* v_pool, int64_t v_row_stride,
                            int Hq, int Dqk, int Dv, const int32_t* q_seq,
                            const int32_t* q_pos, int Nq, const int32_t* idx, int K,
                            float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                            dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Cache write: store new rows into the paged caches -- a whole prompt after
 * prefill, the appended token at each decode step.  Source: "Day-0
 * Adaptation of Ultra-Large-Scale MoE Models on Heterogeneous AI
 * Accelerators", section 4: the KV cache is written in the block layout, and
 * the layout written during prefill must match exactly the gather addresses
 * read during decode.  Row i goes to position pos[i] of sequence seq[i], i.e.
 * physical row block_table[seq][pos / block_size] * block_size
 * + pos % block_size -- the same mapping every gather above uses.
 *
 *  layout      paged layout (seq_lens is read only by the append form)
 *  seq, pos    [N] int32 sequence and position of each new row; both NULL:
 *              the append form of a decode step, row i goes to position
 *              seq_lens[i] - 1 of sequence i (N <= batch; seq_lens already
 *              counts the new token)
 *  kv_new      [N][row_elems] bf16 rows (K, or the latent K/V row), or NULL
 *  row_elems   bf16 elements per row, a multiple of 8
 *  kv_pool     physical rows of row_elems bf16, kv_row_stride elements apart
 *              (a multiple of 8, >= row_elems)
 *  kidx_new    [N][D_i] indexer-key rows of kidx_dtype, or NULL
 *  kidx_pool   [num_blocks][block_size][D_i] of kidx_dtype
 *  ws          workspace of dsa_cache_write_workspace_size() bytes
 * Pointers 16-byte aligned.  Rows of the same physical row written twice in
 * one call (a caller error the call does not detect): each 16-byte piece of
 * that row holds the piece of one of them, which one unspecified, so the row
 * may mix them.
 * Errors: DSA_ERR_INVALID for null pointers, N < 0, bad sizes, strides or
 * alignment.  Device: a sequence outside [0, batch), a position outside the
 * block table or a block id outside [0, num_blocks) skips that row and sets
 * DSA_STATUS_BAD_BLOCK.
 */
size_t dsa_cache_write_workspace_size(void);
int dsa_cache_write(const dsa_paged_layout* layout, const int32_t* seq, const int32_t* pos, int N,
                    const void* kv_new, int row_elems, void* kv_pool, int64_t kv_row_stride,
                    const void* kidx_new, int D_i, int kidx_dtype, void* kidx_pool, void* ws,
                    size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Whole steps: one call for one decode step or one prefill (chunk), each the
 * cache write followed by the three stages on `stream` (no host
 * synchronisation in between).  Source: "Day-0 Adaptation of
 * Trillion-Parameter MoE Models on Domestic GPUs", section 3 (3): decode
 * indexing is incremental -- the indexer keys of earlier positions stay in
 * the cache and a step only adds the new position's row before scoring --
 * and prefill handles a whole prompt at once; "Day-0 Adaptation of
 * Ultra-Large-Scale MoE Models on Heterogeneous AI Accelerators", section 4:
 * index selection, KV cache write, then gather + sparse attention.
 *
 * dsa_decode_step: layout->seq_lens[b] already counts sequence b's new token.
 *  k_new       [B][Dqk] bf16 new K rows (the latent row for a latent cache),
 *              written at position seq_lens[b] - 1 of k_pool (rows
 *              k_row_stride elements apart)
 *  v_new       [B][Dv] bf16 new V rows into v_pool, or NULL when v_pool is
 *              k_pool and V is the first Dv dims of the K row
 *  kidx_new    [B][D_i] new indexer-key rows of idx_dtype into kidx_pool
 *  q_idx, w, q as for dsa_index_score / dsa_sparse_attn_decode (query b is
 *              sequence b at its newest position)
 *  scores      [B][ld], idx [B][K], out [B][Hq][Dv], lse [B][Hq] or NULL
 *  ws          dsa_decode_step_workspace_size(...) bytes; the step's status
 *              word (all stages OR into it) is at offset 0
 * dsa_prefill_step: the Nq queries of sequence `seq` at positions q_pos
 * (device [Nq]); their new rows (k_new/v_new/kidx_new, [Nq][...]) are written
 * at those positions first, so a prompt (or a chunk of one after an existing
 * prefix) is cached and attended in one call; n_eligible [Nq] = q_pos + 1.
 * Errors: those of the calls the step makes, with nothing after the first
 * failing call launched.
 */
size_t dsa_decode_step_workspace_size(int B, int H_i, int D_i, int64_t ld, int Hq, int Dqk,
                                      int Dv, int K);
int dsa_decode_step(const dsa_paged_layout* layout, const void* k_new, void* k_pool,
                    int64_t k_row_stride, const void* v_new, void* v_pool, int64_t v_row_stride,
                    const void* kidx_new, void* kidx_pool, int idx_dtype, const void* q_idx,
                    const float* w, int H_i, int D_i, const void* q, int Hq, int Dqk, int Dv,
                    int K, float sm_scale, float* scores, int64_t ld, int32_t* idx, void* out,
                    float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream);
size_t dsa_prefill_step_workspace_size(int Nq, int H_i, int D_i, int64_t ld, int Hq, int Dqk,
                                       int Dv, int K);
int dsa_prefill_step(const dsa_paged_layout* layout, int seq, const int32_t* q_pos,
                     const int32_t* n_eligible, int Nq, const void* k_new, void* k_pool,
                     int64_t k_row_stride, const void* v_new, void* v_pool, int64_t v_row_stride,
                     const void* kidx_new, void* kidx_pool, int idx_dtype, const void* q_idx,
                     const float* w, int H_i, int D_i, const void* q, int Hq, int Dqk, int Dv,
                     int K, float sm_scale, float* scores, int64_t ld, int32_t* idx, void* out,
                     float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream);

/* dsa_prefill_step_chunked — "Day-0 Adaptation of Trillion-Parameter MoE Models
 * on Domestic GPUs", section 3 (3): the prefill stage fuses index selection and
 * exact attention into large-granularity operators.  The same work as
 * dsa_prefill_step (cache write, indexer score, top-K, attention; same
 * arguments and results), without the [Nq][ld] score matrix: the queries are
 * scored and selected `chunk` rows at a time, and a chunk's scores live in one
 * scratch region of the workspace that the next chunk overwrites.  The score
 * memory is chunk x ld x 4 bytes instead of Nq x ld x 4 (a 16384-token prompt:
 * 48 MB instead of 1 GB), and with the default chunk it stays in L2 between the
 * indexer that writes it and the top-K that reads it, so the scores make no
 * round trip through HBM.
 *  ld          row length of the scratch (>= the largest n_eligible)
 *  chunk       queries per chunk; 0: the largest multiple of 16 whose scores
 *              fit 48 MB (at least 16)
 *  idx, out, lse, ws: as for dsa_prefill_step; ws =
 *              dsa_prefill_step_chunked_workspace_size(...) bytes, for the same
 *              chunk argument
 * Errors: those of dsa_prefill_step; chunk < 0 is DSA_ERR_INVALID.
 */
size_t dsa_prefill_step_chunked_workspace_size(int Nq, int H_i, int D_i, int64_t ld, int Hq,
                                               int Dqk, int Dv, int K, int chunk);
int dsa_prefill_step_chunked(const dsa_paged_layout* layout, int seq, const int32_t* q_pos,
                             const int32_t* n_eligible, int Nq, const void* k_new, void* k_pool,
                             int64_t k_row_stride, const void* v_new, void* v_pool,
                             int64_t v_row_stride, const void* kidx_new, void* kidx_pool,
                             int idx_dtype, const void* q_idx, const float* w, int H_i, int D_i,
                             const void* q, int Hq, int Dqk, int Dv, int K, float sm_scale,
                             int64_t ld, int chunk, int32_t* idx, void* out, float* lse, void* ws,
                             size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Block-level bounds for incremental decode indexing — "Day-0 Adaptation of
 * Trillion-Parameter MoE Models on Domestic GPUs", section 3 (3): decode-time
 * index selection reuses the index structure of earlier steps and computes
 * only what is needed.  The structure is a bound pool beside the indexer-key
 * pool: for every page, per key dimension d, the largest and the smallest key
 * over the page's cached positions, as key codes:
 *   kbound_pool [NB][2][D_i] in the keys' dtype (row 0 maxima, row 1 minima).
 * dsa_index_bounds_update: recompute the bounds of the pages holding the rows
 *   (seq[i], pos[i]), i < N — call it after dsa_cache_write with the same
 *   seq/pos (after a decode step's append: one page per sequence) — or, with
 *   seq = pos = NULL, of every page slot below each sequence's length.  The
 *   layout's seq_lens must include the rows written.  ws: the status word
 *   (dsa_index_bounds_update_workspace_size() bytes); a page id outside
 *   [0, NB) is skipped and flags DSA_STATUS_BAD_BLOCK.
 * dsa_index_score_bounded: the decode form of dsa_index_score (query b is the
 *   query of sequence b, every cached position eligible, B = layout->batch,
 *   scores [B][ld]) that leaves out 128-position tiles whose scores cannot
 *   reach the top-K of size K: the bounds give each tile an upper bound of
 *   its scores; the ceil(K/128) + 1 tiles with the largest bounds are scored
 *   first, and every other tile whose bound is below the K-th largest of
 *   those scores is left out — its scores are -inf, its keys are not read.
 *   Every other score equals dsa_index_score's, so dsa_topk over the row
 *   selects exactly what it selects over the full row.  Pays off only where
 *   pages differ in their keys (on keys drawn independently per position
 *   every bound covers the row's largest score and nothing is left out).
 *   ws: dsa_index_score_bounded_workspace_size(B, H_i, D_i, ld, K) bytes.
 *   B <= 65535 (DSA_ERR_UNSUPPORTED otherwise, nothing launched).
 * dsa_index_bounded_stats: after the work queued on `stream` (this call
 *   synchronises it), the tiles the last dsa_index_score_bounded call on ws
 *   left out and the tiles it bounded.
 */
size_t dsa_index_bounds_update_workspace_size(void);
int dsa_index_bounds_update(const dsa_paged_layout* layout, const int32_t* seq,
                            const int32_t* pos, int N, const void* kidx_pool, int D_i,
                            int idx_dtype, void* kbound_pool, void* ws, size_t ws_bytes,
                            dsa_stream_t stream);
size_t dsa_index_score_bounded_workspace_size(int B, int H_i, int D_i, int64_t ld, int K);
int dsa_index_score_bounded(const dsa_paged_layout* layout, const void* q_idx, const float* w,
                            const void* kidx_pool, int idx_dtype, int H_i, int D_i,
                            const void* kbound_pool, int K, float* scores, int64_t ld, void* ws,
                            size_t ws_bytes, dsa_stream_t stream);
int dsa_index_bounded_stats(void* ws, dsa_stream_t stream, uint64_t* tiles_skipped,
                            uint64_t* tiles_bounded);

/* ---------------------------------------------------------------------------
 * Heads of new tokens: norm and position rotation on the way to where they
 * are read.  The pages start from finished indexer queries, queries and cache
 * rows; these calls make them from a layer's raw projections.  The cache
 * layout is that of "Day-0 Adaptation of Ultra-Large-Scale MoE Models on
 * Heterogeneous AI Accelerators", section 4 (the layout written must match
 * the addresses the gather reads).
 *
 * A part is one tensor of `heads` heads of `dim` elements for each of N
 * tokens.  Each head x[0..dim) is, in fp32,
 *   normed over its first norm_dim elements (the others pass through):
 *     DSA_NORM_RMS    y = x / sqrt(mean(x^2) + eps) * weight + bias
 *     DSA_NORM_LAYER  y = (x - m) / sqrt(mean((x - m)^2) + eps) * weight + bias
 *   rotated in [rope_offset, rope_offset + rope_dim): pair i becomes
 *     (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i],
 *     the pair being elements (2 i, 2 i + 1) if interleaved, else
 *     (i, i + rope_dim / 2) of that range; t is reduced modulo 2 pi in
 *     integers, so it stays exact to ~2e-7 at any position (inv_freq <= 1);
 *   rounded once to out_dtype (E4M3 saturates at +-448).
 * in, out and weights are device pointers.  heads >= 1; dim a multiple of 8,
 * 8..1024; strides in elements, multiples of 8; in and a bf16 out 16-byte
 * aligned, an FP8 out 8-byte; weight and bias 16-byte aligned; rope_offset
 * and rope_dim even.  out may be in itself (bf16, same strides); apart from
 * that no part's out may overlap any part's in or out.
 *
 * All parts of a launch take one code path, the slowest that one of them needs:
 * a norm_dim, or a rotated range or half of one, that is no multiple of 8; a dim
 * beyond 768; dims beyond 256 beside such a rotation; a pair with only one
 * element inside the norm.  Such a part costs the others up to six times their
 * time, and is better given a call of its own where speed counts.
 */
#define DSA_NORM_NONE 0
#define DSA_NORM_RMS 1
#define DSA_NORM_LAYER 2
#define DSA_MAX_HEAD_PARTS 4 /* parts per list */

typedef struct dsa_head_part {
  const void* in;           /* bf16, token t head h at in + t*in_token_stride + h*in_head_stride */
  int64_t in_token_stride;
  int64_t in_head_stride;
  void* out;                /* of out_dtype */
  int64_t out_token_stride; /* elements between tokens; of a pool: between its rows */
  int64_t out_head_stride;
  int32_t out_dtype;        /* DSA_BF16 or DSA_FP8_E4M3 */
  int32_t heads;
  int32_t dim;
  int32_t norm;             /* DSA_NORM_* */
  int32_t norm_dim;         /* 1..dim when norm is not NONE */
  float eps;                /* >= 0 */
  const float* weight;      /* [norm_dim] fp32, or NULL (1) */
  const float* bias;        /* [norm_dim] fp32, or NULL (0) */
  int32_t rope_offset;
  int32_t rope_dim;         /* 0: no rotation */
  int32_t interleaved;
  int32_t reserved_;        /* set to 0 */
  const float* inv_freq;    /* [rope_dim / 2] fp32, finite */
} dsa_head_part;

/* dsa_head_norm_rope: the parts (1..DSA_MAX_HEAD_PARTS tensors, such as the
 * latent queries' rotated part and the indexer queries, or queries and keys)
 * of N tokens at positions pos [N] (device int32), in one launch.  `parts` is
 * a host array, read before the call returns.  pos may be NULL when no part
 * rotates.
 * Errors: DSA_ERR_INVALID for null pointers, N < 0, n_parts, strides or
 * alignment; DSA_ERR_UNSUPPORTED for other dims, dtypes or norms, and for
 * more than 2^31 - 64 (token, head) rows in all.
 */
int dsa_head_norm_rope(const dsa_head_part* parts, int n_parts, const int32_t* pos, int N,
                       dsa_stream_t stream);

/* dsa_cache_append: dsa_cache_write with the transform on the way.  cache
 * parts (1..DSA_MAX_HEAD_PARTS: K or latent rows, V rows, indexer keys) go to
 * physical row block_table[seq][pos / block_size] * block_size
 * + pos % block_size of their pool `out` (rows out_token_stride elements
 * apart, heads out_head_stride apart inside a row); heads parts (0..
 * DSA_MAX_HEAD_PARTS, may be NULL) are the same tokens' queries, written as
 * dsa_head_norm_rope writes them, in the same launch.
 *  seq, pos    [N] int32 sequence and position of each token; both NULL: the
 *              append form of a decode step, token i is position
 *              seq_lens[i] - 1 of sequence i (N <= batch)
 *  ws          dsa_cache_append_workspace_size() bytes (the status word)
 * A token whose sequence, position or page is out of range has its cache rows
 * skipped and sets DSA_STATUS_BAD_BLOCK; its heads parts are still written,
 * rotated by its position.  The same physical row twice in one call: as for
 * dsa_cache_write.  Other errors as for dsa_head_norm_rope.
 */
size_t dsa_cache_append_workspace_size(void);
int dsa_cache_append(const dsa_paged_layout* layout, const int32_t* seq, const int32_t* pos, int N,
                     const dsa_head_part* cache, int n_cache, const dsa_head_part* heads,
                     int n_heads, void* ws, size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * dsa_prefix_attn_decode: exact attention of one query per sequence over all
 * of its cached positions, for a batch that shares a prefix.  Where no more
 * than K positions are eligible the selection keeps every one of them, and
 * this call needs neither scores nor an index list; requests behind one
 * prompt read its pages once for the whole batch.  The result is that of
 * dsa_sparse_attn_decode with every position selected:
 *     z_p = sm_scale * q[b][h] . K_p,  out[b][h] = sum_p softmax(z)_p V_p,
 *     lse[b][h] = log sum_p exp(z_p),  p < seq_lens[b]
 * Scores, maxima and sums are fp32.  The weights enter the product with V as
 * bf16 hi + lo (each off by at most 2^-16 of itself) for a sequence of at most
 * 512 positions, and rounded once to bf16 (at most 2^-8 of itself) for a longer
 * one, as dsa_sparse_attn_decode has them for 64 heads of 576/512 (its other
 * shapes keep fp32 weights).  out is rounded once.
 *  prefix_len  0..max_seq_len: positions [0, prefix_len) hold the same rows
 *              for every sequence with seq_lens[b] >= prefix_len (normally
 *              the same pages; they are read through the block-table row of
 *              the first such sequence).  A shorter sequence shares nothing:
 *              its own pages alone are read.  0: dense decode attention.
 *  q           [B][Hq][Dqk] bf16, B = layout->batch
 *  k_pool, v_pool, strides: as for dsa_sparse_attn_decode (v_pool may be
 *              k_pool); Hq 1..128, Dqk 8..576 and Dv 8..512 multiples of 8
 *  out         [B][Hq][Dv] bf16 (0 for an empty sequence)
 *  lse         [B][Hq] fp32, or NULL (-inf for an empty sequence)
 *  ws          dsa_prefix_attn_decode_workspace_size() bytes
 * A call has one key head.  Rows of several (as dsa_cache_append stores them)
 * take a call per key head: k_pool and v_pool at that head's first element of
 * row 0, the strides those of the whole rows, q and out of its query heads.
 * Errors: DSA_ERR_INVALID / DSA_ERR_UNSUPPORTED as for
 * dsa_sparse_attn_decode, for prefix_len out of range, and for more than 2^30
 * tiles of 128 rows x 256 positions.  Device: a position behind a bad block id
 * is left out and sets DSA_STATUS_BAD_BLOCK; a length beyond max_seq_len is
 * cut there and sets DSA_STATUS_BAD_LENGTH; a bounded wait that ran out sets
 * DSA_STATUS_TIMEOUT (the outputs are then not valid).
 */
size_t dsa_prefix_attn_decode_workspace_size(int B, int Hq, int Dqk, int Dv, int prefix_len);
int dsa_prefix_attn_decode(const dsa_paged_layout* layout, const void* q, const void* k_pool,
                           int64_t k_row_stride, const void* v_pool, int64_t v_row_stride, int Hq,
                           int Dqk, int Dv, int prefix_len, float sm_scale, void* out, float* lse,
                           void* ws, size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * dsa_prompt_attn: exact causal attention of whole prompts, or of chunks behind
 * keys that are in hand, several sequences packed end to end, grouped heads.
 * The first pages' prefill selects keys; this call is for layers, or prompts no
 * longer than the selection, that attend every one of them.  Token i of the nq
 * query tokens of a sequence with nk keys sees keys j <= i + nk - nq (the last
 * token sees all):
 *     z_j = sm_scale * q[i][h] . k[j][h'],  out[i][h] = sum_j softmax(z)_j v[j][h'],
 *     lse[i][h] = log sum_j exp(z_j),  h' = h / (Hq / Hk)
 * A token that sees no key (nk < nq) has out 0 and lse -inf. Scores, maxima and
 * sums are fp32 (the matrix unit's own run over 2^18 keys at most). A weight
 * enters the product with V as bf16, off by at most 2^-8 of itself, and as bf16
 * hi + lo (2^-16) for the tokens whose tile begins with one that sees no more
 * than 512 keys; out is rounded once. The single rounding of the weights adds
 * about as much to the error of out as its own rounding does (0.0023 of its norm
 * instead of 0.0017 behind 6,000 keys), in exchange for a third of the matrix
 * work. What a token does not see does not reach it, NaN and infinities included.
 *  q, k, v     bf16: token i head h at ptr + i * token stride + h * head stride
 *              (elements, multiples of 8, heads not overlapping); q has Nq tokens
 *              and Hq heads, k and v Nk tokens and Hk heads; 16-byte aligned
 *  cu_q, cu_k  device int32 [B + 1], not decreasing: sequence b has query tokens
 *              cu_q[b] .. cu_q[b + 1] - 1 and keys cu_k[b] .. cu_k[b + 1] - 1;
 *              NULL (with B = 1): all of them.  Tokens of no sequence are not
 *              written.
 *  Hq, Hk      Hq a multiple of Hk;  Dk, Dv multiples of 8, 8..256
 *  out         bf16 [Nq][Hq][Dv] with strides like q's;  lse [Nq][Hq] fp32 or NULL.
 *              May not overlap q, k or v: an item writes its tokens while others
 *              still read them.
 *  ws          dsa_prompt_attn_workspace_size() bytes: 72 MB of partial results
 *              and sums, the same for every call, so that a workspace asked for
 *              once serves longer and shorter ones
 * Errors: DSA_ERR_INVALID for null pointers, strides, alignment or sm_scale;
 * DSA_ERR_UNSUPPORTED for other heads and dims and beyond 2^31 items of 256 rows.
 * Device: a sequence whose offsets are not inside the tokens is left out and sets
 * DSA_STATUS_BAD_LENGTH; a bounded wait that ran out sets DSA_STATUS_TIMEOUT (the
 * outputs are then not valid).
 */
size_t dsa_prompt_attn_workspace_size(int B, int Nq, int Hq, int Hk, int Dk, int Dv);
int dsa_prompt_attn(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                    int64_t k_token_stride, int64_t k_head_stride, const void* v,
                    int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                    const int32_t* cu_k, int B, int Nq, int Nk, int Hq, int Hk, int Dk, int Dv,
                    float sm_scale, void* out, int64_t out_token_stride, int64_t out_head_stride,
                    float* lse, void* ws, size_t ws_bytes, dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * A K/V cache held in 4 bits, for grouped heads.  The pages are those of the
 * layout; what a page holds is the calls' own:
 *   pool  uint8 [num_blocks][Hk][block_size][row bytes], 16-byte aligned, row
 *         bytes = dsa_cache4_row_bytes(Dk, Dv) (0 for unsupported dims).
 * A row is one position of one key head: Dk / 2 bytes of K codes, Dv / 2 of V
 * codes (two E2M1 codes a byte, the lower dim in the lower half), one E4M3
 * scale per 16 dims of K, then of V, and zeros up to a multiple of 16 bytes.
 * A code c stands for  head scale * group scale * c.  A group of 16 elements
 * y = x / head scale is kept as
 *     group scale s = E4M3(min(max |y| / 6, 448)),  c = E2M1 nearest to y / s
 * (y rounded to fp32; ties to the even code; codes are 0 where s is 0 or NaN).
 * An infinity is kept as +-2688 head scales, a NaN makes its whole group NaN.
 *  Hk, Dk, Dv  Hk >= 1; Dk and Dv multiples of 16, 16..256
 *  k_scale, v_scale  [Hk] fp32 head scales, finite and positive, or NULL (1)
 */
size_t dsa_cache4_row_bytes(int Dk, int Dv);

/* dsa_cache4_write: K and V rows of N new tokens into the pool.
 *  seq, pos    as for dsa_cache_append: [N] int32, or both NULL (token i is
 *              position seq_lens[i] - 1 of sequence i, N <= batch)
 *  k, v        bf16, token i head h at ptr + i * token stride + h * head
 *              stride; 16-byte aligned, strides in elements, multiples of 8,
 *              not negative
 *  k_out, v_out  [N][Hk][Dk] and [N][Hk][Dv] bf16, 16-byte aligned, both or
 *              neither: the values that the cache keeps, rounded to bf16 (exact
 *              where the head scale is 1), for an attention of the prompt that
 *              sees what later steps will see.  May not overlap k or v.
 *  ws          dsa_cache4_write_workspace_size() bytes (the status word)
 * A token whose sequence, position or page is out of range is not stored and
 * sets DSA_STATUS_BAD_BLOCK; its k_out and v_out are written all the same.  The
 * same position twice in one call (a caller error the call does not detect): each
 * byte of its rows comes from one of the two, which one unspecified, so that a
 * group may get the codes of one and the scale of the other.
 * Rows that no token names keep every byte.
 * Errors: DSA_ERR_INVALID for null pointers, N, strides or alignment;
 * DSA_ERR_UNSUPPORTED for other dims, for N * Hk beyond 2^31 - 1 and for
 * Hk * (Dk + Dv) beyond 2^33.
 */
size_t dsa_cache4_write_workspace_size(void);
int dsa_cache4_write(const dsa_paged_layout* layout, const int32_t* seq, const int32_t* pos, int N,
                     const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v,
                     int64_t v_token_stride, int64_t v_head_stride, int Hk, int Dk, int Dv,
                     const float* k_scale, const float* v_scale, void* pool, void* k_out,
                     void* v_out, void* ws, size_t ws_bytes, dsa_stream_t stream);

/* dsa_cache4_read: the values of N positions of the pool as bf16 heads, such as
 * a cached prefix for the dsa_prompt_attn of the chunk behind it.
 *  seq, pos    [N] int32, both given
 *  k_out, v_out  [N][Hk][Dk] and [N][Hk][Dv] bf16, 16-byte aligned
 * A token out of range reads as zeros and sets DSA_STATUS_BAD_BLOCK.  Errors as
 * for dsa_cache4_write.
 */
size_t dsa_cache4_read_workspace_size(void);
int dsa_cache4_read(const dsa_paged_layout* layout, const int32_t* seq, const int32_t* pos, int N,
                    int Hk, int Dk, int Dv, const float* k_scale, const float* v_scale,
                    const void* pool, void* k_out, void* v_out, void* ws, size_t ws_bytes,
                    dsa_stream_t stream);

/* dsa_cache4_attn_decode: exact attention of one query per sequence over all of
 * its positions in the 4-bit pool: for query head h over key head h / (Hq / Hk)
 *     z_p = sm_scale * q[b][h] . K_p,  out[b][h] = sum_p softmax(z)_p V_p,
 *     lse[b][h] = log sum_p exp(z_p),  p < seq_lens[b]
 * on the values that the codes stand for.  Scores, maxima and sums are fp32; a
 * weight enters the product with V as fp16, off by at most 2^-11 of itself, or by
 * 2^-32 of the row's largest weight; out is rounded once.
 *  q           [B][Hq][Dk] bf16, B = layout->batch, Hq a multiple of Hk
 *  out         [B][Hq][Dv] bf16 (0 for an empty sequence); may not overlap q
 *  lse         [B][Hq] fp32, or NULL (-inf for an empty sequence)
 *  ws          dsa_cache4_attn_decode_workspace_size() bytes
 * Errors: DSA_ERR_INVALID for null pointers, alignment (q, pool and out 16
 * bytes) or sm_scale; DSA_ERR_UNSUPPORTED for other dims, Hq no multiple of Hk,
 * and beyond 2^31 units of 256 positions.  Device: a position behind a bad block
 * id is left out and sets DSA_STATUS_BAD_BLOCK; a length beyond max_seq_len is
 * cut there and sets DSA_STATUS_BAD_LENGTH; a bounded wait that ran out sets
 * DSA_STATUS_TIMEOUT (the outputs are then not valid).
 */
size_t dsa_cache4_attn_decode_workspace_size(int B, int Hq, int Hk, int Dk, int Dv);
int dsa_cache4_attn_decode(const dsa_paged_layout* layout, const void* q, const void* pool, int Hq,
                           int Hk, int Dk, int Dv, const float* k_scale, const float* v_scale,
                           float sm_scale, void* out, float* lse, void* ws, size_t ws_bytes,
                           dsa_stream_t stream);

/* ---------------------------------------------------------------------------
 * Utilities (no counterpart on the pages).
 * dsa_get_status: copy the status word of a workspace to *status (host), after
 *   the work queued on `stream` so far has finished (this call synchronises the
 *   stream); clear != 0 resets it to 0.  Returns DSA_OK or DSA_ERR_*.
 * dsa_last_error_string: message of the last failing call on this host thread.
 * dsa_launch_count: kernels this library has launched in this process.
 * dsa_version: 10000*major + 100*minor + patch.
 * dsa_selftest_bounded_wait: one bounded mbarrier wait of the kind every
 *   pipelined kernel uses (one thread of one CTA).  expire != 0: nothing
 *   arrives, the wait gives up after limit_ns (1 us .. 1 s) and
 *   DSA_STATUS_TIMEOUT is OR-ed into the status word of ws (>= 256 bytes);
 *   expire == 0: the barrier completes first and nothing is recorded.  For
 *   testing the give-up path without a hang; the context stays usable.
 * dsa_selftest_warp_wait: the same for the whole-warp wait of
 *   dsa_prefix_attn_decode.  mode 0: the barrier completes first; 1: nothing
 *   arrives; 2: nothing arrives and another warp raises the kernel's abort flag
 *   after 5 ms, which ends the wait before its limit.  Modes 1 and 2 set
 *   DSA_STATUS_TIMEOUT.
 */
int dsa_get_status(void* ws, dsa_stream_t stream, int32_t* status, int clear);
const char* dsa_last_error_string(void);
uint64_t dsa_launch_count(void);
int dsa_version(void);
int dsa_selftest_bounded_wait(int expire, uint64_t limit_ns, void* ws, size_t ws_bytes,
                              dsa_stream_t stream);
int dsa_selftest_warp_wait(int mode, uint64_t limit_ns, void* ws, size_t ws_bytes,
                           dsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_H_ */
