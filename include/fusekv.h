/*
 * fusekv.h -- C ABI of the cache-fusion layer-step library (libfusekv.so).
 *
 * One layer-step of RAG KV-cache fusion with selective recomputation, as
 * stated on two pages:
 *   [QCFuse]  "QCFuse: Query-Aware Cache Fusion via Compressed View for
 *             Efficient RAG Serving", section 2.1 (Eqs. 1-7), Eq. 11,
 *             section 3.2.1 (Eqs. 9-10), section 3.4.2 (Eq. 20).
 *   [KVBoost] "KVBoost: Chunk-Level KV Cache Reuse with Deviation-Guided
 *             Recomputation", sections 3.1-3.2 (Eqs. 1-3), 4.5 (Eq. 7),
 *             4.6.2 (Alg. 2, CacheBlendRecompute).
 *   [PCR]     "PCR: A Prefetch-Enhanced Cache Reuse System for Low-Latency
 *             RAG Serving", layer-wise overlapping (Figure 8).
 *
 * Conventions shared by every call
 * --------------------------------
 * Ownership.  The caller allocates and owns every buffer, the workspace
 *   included.  The library allocates no device memory and keeps no pointer
 *   after a call returns.  All work is enqueued on the caller's stream; the
 *   buffers must stay valid until the stream has passed that point.
 * Pointers.  Every tensor pointer is a device pointer aligned to 16 bytes,
 *   unless the field says "host".
 * Errors.  Argument errors are detected on the host and returned before any
 *   launch; every call that takes a request table rejects one of more
 *   than 65535 requests with FUSE_ERR_UNSUPPORTED.  Launch failures return
 *   FUSE_ERR_CUDA.  Errors that only the GPU can see (an out-of-range block
 *   id or selected index, an unsorted index list, a wait that timed out)
 *   are recorded in the workspace's error word
 *   and reported by fuse_check_errors().  Nothing aborts or exits.
 * Layouts (row-major, innermost last).
 *   H        [T_total, hidden]            current hidden states; request r owns
 *                                         rows [row0, row0 + N_r + Qn_r): its N_r
 *                                         context tokens, then its Qn_r query tokens.
 *   Wq       [Hq * d, hidden]             projection weights (nn.Linear layout:
 *   Wk, Wv   [Hkv * d, hidden]             out x in, both GEMM operands K-major).
 *   Kf, Vf   [T_total, Hkv, d]            the fused cache, rows aligned with H.
 *   score    [N_total]                    request r's scores at [score0, score0 + N_r).
 *   idx      [K_total] int32              request r's k_r selected context
 *                                         positions (request-local, ascending) at
 *                                         [sel0, sel0 + k_r).
 *   O        [R_total, Hq, d]             attention rows of S_r = idx_r U {N_r .. T_r-1}
 *                                         in ascending position, at [out0, out0 + R_r),
 *                                         R_r = k_r + Qn_r.
 *   Query head h reads KV head h / (Hq / Hkv).  Positions are request-local:
 *   context token t sits at position t, query token j at N_r + j.
 * RoPE.  Rotate-half pairing (j, j + d/2) with theta_j = base^(-2j/d); the
 *   rotation R^p turns pair j by the angle p * theta_j ([KVBoost] Eq. 3).
 */
#ifndef FUSEKV_H
#define FUSEKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream (cudaStream_t); NULL is the legacy default stream. */
typedef struct CUstream_st* fuse_stream_t;

typedef enum {
  FUSE_OK = 0,
  FUSE_ERR_INVALID_ARG = 1,   /* null pointer, bad size, inconsistent tables      */
  FUSE_ERR_MISALIGNED = 2,    /* a pointer or row stride not aligned to 16 bytes   */
  FUSE_ERR_UNSUPPORTED = 3,   /* a valid request the library does not handle       */
  FUSE_ERR_WORKSPACE = 4,     /* workspace null or smaller than fuse_workspace_size */
  FUSE_ERR_CUDA = 5,          /* a CUDA runtime call or launch failed              */
  FUSE_ERR_TIMEOUT = 6,       /* (device) a bounded wait gave up                   */
  FUSE_ERR_DEVICE_BOUNDS = 7, /* (device) an index read from device memory was out
                                 of range or out of order; the access was skipped  */
  FUSE_ERR_NO_PAGES = 8       /* (device) a pool has too few free pages; nothing changed */
} fuse_status_t;

typedef enum { FUSE_F32 = 0, FUSE_BF16 = 1, FUSE_U8_ASYM = 2, FUSE_U4_ASYM = 3 } fuse_dtype_t;
typedef enum { FUSE_KV_CONTIGUOUS = 0, FUSE_KV_PAGED = 1 } fuse_kv_layout_t;
typedef enum { FUSE_ROPE_ROTATE_HALF = 0 } fuse_pos_encoding_t;

/* Shape of one attention layer.  head_dim must be 64 or 128 and n_q_heads a
 * multiple of n_kv_heads.  dtype (FUSE_F32 or FUSE_BF16) is the storage type
 * of H, the weights, the fused cache, Q and O; arithmetic accumulates in fp32.
 * Only rotary position encoding is accepted ([KVBoost] section 5 limits reuse
 * to RoPE models): any other pos_encoding returns FUSE_ERR_UNSUPPORTED. */
typedef struct {
  int32_t hidden;
  int32_t n_q_heads;
  int32_t n_kv_heads;
  int32_t head_dim;
  double rope_base;
  int32_t pos_encoding;
  int32_t dtype;
} fuse_layer_desc_t;

/* One cached chunk c_i of a request ([QCFuse] Eqs. 1, 3): its keys were
 * computed alone at chunk-local positions 0 .. len-1.
 *   dst_row  first row of the chunk in the packed fused cache / H.
 *   pos      request-local position o_i of the chunk's first token (the
 *            re-rotation angle offset, [QCFuse] Eq. 4).
 *   len      number of tokens.
 * Storage, selected by fuse_chunks_t.kv_layout / kv_storage:
 *   CONTIGUOUS  k, v point at this chunk's own [len, Hkv, d] arrays.
 *   PAGED       k, v point at the shared pool [n_blocks, block_size, Hkv, d];
 *               block_table (device, [ceil(len / block_size)] int32) lists the
 *               pool blocks holding tokens 0.., block_size per block.
 *   U8_ASYM     KIVI asymmetric int8 ([KVBoost] Eq. 7), codes uint8 0..255,
 *               x = zero + q * scale with fp16 scale and zero:
 *               k_scale, k_zero  [Hkv, d]  per channel over the chunk's tokens;
 *               v_scale, v_zero  [len, Hkv] per token (CONTIGUOUS) or
 *                                [n_blocks, block_size, Hkv] (PAGED pool).
 *   U4_ASYM     the same with 4-bit codes 0..15 (KIVI's b = 4), two per byte:
 *               element 2m of a row in the low nibble of byte m, 2m + 1 in
 *               the high nibble, so k and v arrays (and the pool) hold d / 2
 *               bytes per (token, head); scale and zero as for U8_ASYM.
 *   For fuse_pic_precompute, k and v are outputs (CONTIGUOUS F32/BF16 only). */
typedef struct {
  const void* k;
  const void* v;
  const int32_t* block_table;
  const void* k_scale;
  const void* k_zero;
  const void* v_scale;
  const void* v_zero;
  int64_t dst_row;
  int32_t pos;
  int32_t len;
} fuse_chunk_t;

/* The chunk table of a call: the same n_chunks entries twice, once in host
 * memory (validated and used to size the grid) and once in device memory
 * (read by the kernels).  The two copies must be identical. */
typedef struct {
  int32_t n_chunks;
  int32_t kv_layout;        /* fuse_kv_layout_t */
  int32_t kv_storage;       /* fuse_dtype_t of the chunk caches */
  int32_t block_size;       /* PAGED: tokens per pool block (> 0) */
  int64_t n_pool_blocks;    /* PAGED: pool size in blocks, for bounds checks */
  const fuse_chunk_t* h_chunks;   /* host   [n_chunks] */
  const fuse_chunk_t* d_chunks;   /* device [n_chunks] */
} fuse_chunks_t;

/* One request of a batch.  fuse_plan_requests() fills these offsets for the
 * packed layouts described at the top of this file. */
typedef struct {
  int64_t row0;     /* first row of the request in H, Kf, Vf            */
  int64_t score0;   /* first entry of its N_r scores in score[]          */
  int64_t sel0;     /* first entry of its k_r selected indices in idx[]  */
  int64_t out0;     /* first row of its R_r = k_r + Qn_r rows in O       */
  int32_t n_ctx;    /* N_r context tokens                                 */
  int32_t n_query;  /* Qn_r query tokens (always recomputed, never scored) */
  int32_t k;        /* k_r selected context tokens, 0 <= k_r <= N_r        */
  int32_t reserved; /* must be 0 */
} fuse_request_t;

/* The request table of a call, host and device copies (identical). */
typedef struct {
  int32_t n_req;
  const fuse_request_t* h_req;   /* host   [n_req] */
  const fuse_request_t* d_req;   /* device [n_req] */
} fuse_requests_t;

/* Totals of a request table (filled by fuse_plan_requests). */
typedef struct {
  int64_t n_tok;    /* T_total = sum (N_r + Qn_r): rows of H, Kf, Vf */
  int64_t n_ctx;    /* N_total: entries of score[] */
  int64_t n_sel;    /* K_total = sum k_r: entries of idx[] */
  int64_t n_out;    /* R_total = sum (k_r + Qn_r): rows of O */
  int32_t max_ctx;  /* max N_r */
  int32_t max_tok;  /* max N_r + Qn_r */
} fuse_totals_t;

/* ---------------------------------------------------------------------- */

/* Number of recomputed context tokens for ratio rho = |P| / N ([QCFuse]
 * Eq. 6): floor(rho * n_ctx + 1e-9), clamped to [0, n_ctx].  The epsilon
 * keeps products such as 0.29 * 100 = 28.999999999999996 from losing a
 * token.  Host function. */
int64_t fuse_k_from_ratio(double ratio, int64_t n_ctx);

/* Host helper: lay requests out back to back.  n_ctx, n_query: host arrays
 * [n_req].  Writes out[n_req] (k_r = fuse_k_from_ratio(ratio, N_r)) and, if
 * totals is not NULL, the totals.  Returns FUSE_ERR_INVALID_ARG on a
 * negative size or a total beyond 2^31 - 1 rows. */
fuse_status_t fuse_plan_requests(int32_t n_req, const int32_t* n_ctx, const int32_t* n_query,
                                 double ratio, fuse_request_t* out, fuse_totals_t* totals);

/* Workspace bytes needed by every call below for the given request table
 * (host copy read) and layer shape.  The workspace is caller-owned device
 * memory, 256-byte aligned, zero-filled before its first use (for example by
 * fuse_workspace_reset) and reusable across calls on one stream; calls on
 * different streams need their own.  It begins with the error word that
 * fuse_check_errors() reads; the rest is scratch that every call writes
 * before it reads. */
fuse_status_t fuse_workspace_size(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                  size_t* bytes);

/* Zero-fill the whole workspace (enqueued on the stream): before its first
 * use, and after a call that recorded a device error. */
fuse_status_t fuse_workspace_reset(void* ws, size_t ws_bytes, fuse_stream_t stream);

/* Position remapping and stitching, [QCFuse] Eq. 4 with the RoPE correction
 * of [KVBoost] section 3.2: for every chunk i and local row r < len_i,
 *   Kf[dst_row_i + r] = R^{pos_i} K_i[r]     (keys re-rotated by the offset)
 *   Vf[dst_row_i + r] = V_i[r]               (values copied in token order)
 * after dequantisation when kv_storage is FUSE_U8_ASYM or FUSE_U4_ASYM
 * ([KVBoost] Eq. 7).
 * A chunk with pos 0 whose storage type equals desc->dtype is copied bit for
 * bit.  Kf, Vf: [fused_rows, Hkv, d] in desc->dtype; every chunk must satisfy
 * dst_row + len <= fused_rows.  Query rows are not touched. */
fuse_status_t fuse_stitch_rerotate(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                                   void* Kf, void* Vf, int64_t fused_rows,
                                   void* ws, size_t ws_bytes, fuse_stream_t stream);

/* Deviation score of every context token ([KVBoost] Alg. 2 step 2, taken on
 * the values of one layer): with Vn = H_t W_V^T split into Hkv heads,
 *   score_t = 1 - (1/Hkv) sum_h cos(Vn[t,h], Vf[t,h]),
 * the cosine's denominator clamped at 1e-30.  Reads H and Vf at the context
 * rows of each request (Vf holds the stitched cached values); writes
 * score[score0 + t] in fp32.  Deterministic: no floating-point atomics. */
fuse_status_t fuse_score_deviation(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                   const void* H, const void* Wv, const void* Vf, float* score,
                                   void* ws, size_t ws_bytes, fuse_stream_t stream);

/* Key deviation, one layer's term of [KVBoost] Alg. 2 step 2 as printed,
 *   delta_t = 1 - (1/(L Hkv)) sum_{l,h} cos(K~_t^(l,h), K_t^(l,h)),
 * which is the mean over the L layers of 1 - (1/Hkv) sum_h cos.  For every
 * context token t of every request, with the fresh key at the token's
 * request position (where the probe pass puts it),
 *   K~_t = R^t W_K x_t  (x_t = H[row0 + t]),   K_t = Kf[row0 + t] (stitched),
 *   v_t  = weight * (1 - (1/Hkv) sum_h cos(K~_t[h], K_t[h])),
 * each cosine's denominator clamped at 1e-30; accumulate == 0 writes v_t to
 * score[score0 + t], accumulate != 0 adds it.  One call per layer with
 * weight = 1/L (the first with accumulate == 0) leaves delta_t in score.
 * The fresh keys are materialised in desc->dtype (a bf16 layer rounds them
 * to bf16); cosines and sums are fp32, heads summed in order, no atomics.
 * Kf and H are only read.  Needs the workspace of fuse_workspace_size.
 * FUSE_ERR_INVALID_ARG for a weight that is not finite. */
fuse_status_t fuse_score_key_deviation(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                       const void* H, const void* Wk, const void* Kf, float weight,
                                       int32_t accumulate, float* score, void* ws,
                                       size_t ws_bytes, fuse_stream_t stream);

/* Query-aware importance of every context token ([QCFuse] section 3.2.1,
 * Eqs. 9-10, the full-view attention mass; section 3.4.2, Eq. 20, its sum
 * over the critical layers).  For request r with N = N_r context and
 * Qn = Qn_r query tokens, query token u (row row0 + N + u of H) has the state
 *   q_{u,h} = R^{N+u} W_Q x_u        (head h, the recomputation's projection)
 * and the score of context token t is the attention weight it receives,
 *   I(t) = sum_{u < Qn} sum_h softmax_{t' < N}(q_{u,h} . Kf[row0 + t', h/g] / sqrt(d))[t],
 * the softmax over the N context keys of the layer's fused cache (Kf after
 * fuse_stitch_rerotate: the PIC keys of [QCFuse] Eq. 4).  Every (u, h)
 * spreads a total of 1, so the scores of a request sum to Qn * Hq.
 * accumulate == 0 writes I to score[score0 + t]; accumulate != 0 adds it
 * (call once per critical layer for Eq. 20's sum).  Kf and H are only read.
 * Query states are materialised in desc->dtype (bf16 layers round q to
 * bf16); logits, weights and sums are fp32.  Deterministic: no
 * floating-point atomics.  Needs the workspace of fuse_workspace_size. */
fuse_status_t fuse_score_attention_mass(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                        const void* H, const void* Wq, const void* Kf,
                                        int32_t accumulate, float* score, void* ws,
                                        size_t ws_bytes, fuse_stream_t stream);

/* TopK(score, k_r) per request ([QCFuse] Eq. 11; [KVBoost] Alg. 2 step 3):
 * the k_r largest scores, ties broken toward the lower token index, -0 equal
 * to +0, written as ascending request-local indices to idx[sel0 ..].  A NaN
 * score is recorded as FUSE_ERR_DEVICE_BOUNDS (it ranks below every number). */
fuse_status_t fuse_select_topk(const fuse_requests_t* reqs, const float* score, int32_t* idx,
                               void* ws, size_t ws_bytes, fuse_stream_t stream);

/* Selective recomputation, [QCFuse] Eqs. 6-7 with [KVBoost] Eqs. 1-3.  For
 * every request and every row s of S_r = idx_r U {N_r .. T_r - 1}:
 *   q = R^s W_Q x_s,  k = R^s W_K x_s,  v = W_V x_s     (x_s = H[row0 + s])
 *   Kf[row0 + s] = k,  Vf[row0 + s] = v                 (scatter, Eq. 7)
 * and, after all scatters, the causal attention row
 *   O[s, h] = softmax_j(q_h . Kf[j, h/g] / sqrt(d)) Vf[j, h/g],  j <= s,
 * over the fused cache (unselected j hold reused entries, selected j the
 * refreshed ones).  idx must be ascending and < N_r (checked on the device). */
fuse_status_t fuse_recompute_selected(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                      const void* H, const void* Wq, const void* Wk,
                                      const void* Wv, const int32_t* idx, void* Kf, void* Vf,
                                      void* O, void* ws, size_t ws_bytes, fuse_stream_t stream);

/* One whole layer-step: fuse_stitch_rerotate, then (if score_this_layer)
 * fuse_score_deviation and fuse_select_topk writing idx, then
 * fuse_recompute_selected reading idx -- the order of [KVBoost] Alg. 2
 * (probe, deviation, select, patch) on the cache of [QCFuse] Eq. 4.  With
 * score_this_layer == 0, idx is an input (a selection made at another layer)
 * and score is not touched (may be NULL).  Kf, Vf have reqs' T_total rows. */
fuse_status_t fuse_layer_step(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                              const fuse_requests_t* reqs, const void* H, const void* Wq,
                              const void* Wk, const void* Wv, int32_t score_this_layer,
                              int32_t* idx, void* Kf, void* Vf, void* O, float* score,
                              void* ws, size_t ws_bytes, fuse_stream_t stream);

/* The buffers of one layer of a stack (every pointer as in fuse_layer_step;
 * chunks points at this layer's chunk table, in host memory). */
typedef struct {
  const fuse_chunks_t* chunks;
  const void* H;
  const void* Wq;
  const void* Wk;
  const void* Wv;
  void* Kf;
  void* Vf;
  void* O;
} fuse_layer_io_t;

/* A stack of n_layers attention layers sharing one selection ([QCFuse]
 * section 3.4 scores critical layers only; the selection is made at one
 * layer and reused by every layer): the scoring layer is stitched, scored
 * and its top-k written to idx first; then every layer l = 0 .. n_layers-1
 * is stitched (the scoring layer only once) and recomputed with that idx.
 * layers: host array [n_layers]; all layers share desc and reqs; score
 * receives the scoring layer's scores.  One workspace serves every layer
 * (the calls run in stream order). */
fuse_status_t fuse_stack_step(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                              int32_t n_layers, int32_t score_layer, const fuse_layer_io_t* layers,
                              int32_t* idx, float* score, void* ws, size_t ws_bytes,
                              fuse_stream_t stream);

/* The same stack as one CUDA graph ([QCFuse] section 3.5: the layers of a
 * fusion step run back to back; a graph replays their launches without the
 * host issuing each one).  fuse_stack_graph_create captures fuse_stack_step
 * with these arguments on `stream` (not the legacy NULL stream, and not a
 * stream already being captured) and instantiates it; fuse_graph_launch
 * replays it on any stream, with every pointer, table and size as captured
 * (the buffers' contents may change between replays; their addresses and
 * the request and chunk tables may not).  A replay computes what the eager
 * call computes, bit for bit.  Argument errors of the captured call are
 * returned by create; no kernel runs during create.  Keep no kernel trace
 * open while creating.  fuse_graph_destroy releases the graph (host-side
 * state; call it after the last replay has been enqueued). */
typedef struct fuse_graph_st* fuse_graph_t;
fuse_status_t fuse_stack_graph_create(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                      int32_t n_layers, int32_t score_layer,
                                      const fuse_layer_io_t* layers, int32_t* idx, float* score,
                                      void* ws, size_t ws_bytes, fuse_stream_t stream,
                                      fuse_graph_t* out);
fuse_status_t fuse_graph_launch(fuse_graph_t graph, fuse_stream_t stream);
void fuse_graph_destroy(fuse_graph_t graph);

/* ---------------------------------------------------------------------- */
/* Layer-wise loading overlapped with the layers' fusion ([QCFuse] Figure 9,
 * pipeline cache fusion: each layer starts from its loaded PIC entries while
 * later layers' caches are still loading; [PCR] layer-wise overlapping,
 * Figure 8: computation starts once the first layer's cache is loaded).     */

/* One host-to-device copy: `bytes` from host memory `src` to device memory
 * `dst`.  The copy overlaps kernels only when `src` is page-locked. */
typedef struct {
  void* dst;
  const void* src;
  size_t bytes;
} fuse_copy_t;

/* The uploads of one layer of a streamed stack: the copies that fill its
 * staging slot (the device buffers its chunk table points into, and any
 * other input the caller streams through the slot). */
typedef struct {
  int32_t slot;                /* 0 .. n_slots - 1 */
  int32_t n_copies;
  const fuse_copy_t* copies;   /* host [n_copies] */
} fuse_layer_upload_t;

/* fuse_stack_step with every layer's inputs uploaded into a ring of n_slots
 * staging slots on copy_stream while earlier layers compute on stream.
 * Layers run in the order: score_layer (stitch, score, select, recompute),
 * then every other layer in index order (stitch, recompute).  The layers
 * share only the selection, so every output equals fuse_stack_step's on the
 * uploaded data.  Layer l's copies start after every earlier layer that
 * used the same slot has finished on stream; layer l's kernels start after
 * its copies.  Every copy also follows all work enqueued on stream before
 * the call (an earlier call's kernels may still read the slots), and the
 * call's last kernel on stream follows every copy, so back-to-back calls on
 * one stream need no ordering by the caller.  With n_slots >= 2 one layer's
 * upload overlaps the previous layer's kernels.  The schedule is the one
 * fuse_stack_pipeline_plan returns.  The call creates and destroys its own
 * CUDA events (2 * n_slots + 1, n_slots <= 64); everything else is as for
 * fuse_stack_step.  copy_stream
 * and stream must differ for any overlap (the same stream runs everything
 * in order).  Argument errors are returned before any copy or launch. */
fuse_status_t fuse_stack_step_streamed(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                       int32_t n_layers, int32_t score_layer,
                                       const fuse_layer_io_t* layers,
                                       const fuse_layer_upload_t* uploads, int32_t n_slots,
                                       fuse_stream_t copy_stream, int32_t* idx, float* score,
                                       void* ws, size_t ws_bytes, fuse_stream_t stream);

/* The operations of a streamed stack, in issue order. */
typedef enum {
  FUSE_OP_WAIT_FREE = 0,    /* copy stream waits until the slot's last user finished  */
  FUSE_OP_COPY = 1,         /* copy stream: the layer's uploads                        */
  FUSE_OP_MARK_READY = 2,   /* copy stream: the slot's data is in place               */
  FUSE_OP_WAIT_READY = 3,   /* compute stream waits for the slot's data               */
  FUSE_OP_COMPUTE = 4,      /* compute stream: the layer's kernels                      */
  FUSE_OP_MARK_FREE = 5     /* compute stream: the layer is done with the slot          */
} fuse_pipeline_op_kind_t;

typedef struct {
  int32_t kind;    /* fuse_pipeline_op_kind_t */
  int32_t layer;
  int32_t slot;
} fuse_pipeline_op_t;

/* The schedule of fuse_stack_step_streamed (host only, no CUDA call):
 * slot_of_layer[l] in 0 .. n_slots-1 for every layer.  Writes at most
 * max_ops operations to ops and their count to *n_ops (5 per layer, plus a
 * FUSE_OP_WAIT_FREE before every reuse of a slot); FUSE_ERR_WORKSPACE when
 * max_ops is too small (*n_ops then holds the count needed). */
fuse_status_t fuse_stack_pipeline_plan(int32_t n_layers, int32_t score_layer,
                                       const int32_t* slot_of_layer, int32_t n_slots,
                                       fuse_pipeline_op_t* ops, int32_t max_ops, int32_t* n_ops);

/* Position-independent chunk caches, [QCFuse] Eq. 3 with one projection layer
 * standing in for the model: for every chunk i and local row r,
 *   K_i[r] = R^r W_K x,  V_i[r] = W_V x,   x = H_clean[dst_row_i + r].
 * This prepares inputs for the calls above (it is not part of a layer-step).
 * Chunk storage must be CONTIGUOUS and equal to desc->dtype. */
fuse_status_t fuse_pic_precompute(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                                  const void* H_clean, const void* Wk, const void* Wv,
                                  void* ws, size_t ws_bytes, fuse_stream_t stream);

/* KIVI asymmetric quantisation of chunk caches ([KVBoost] section 4.5,
 * Eq. 7, b = 8 for FUSE_U8_ASYM, b = 4 for FUSE_U4_ASYM), the inverse of the
 * stitch's dequantisation; it prepares int8 / int4 inputs (it is not part of
 * a layer-step).  src: CONTIGUOUS caches in desc->dtype; dst: CONTIGUOUS
 * with the same n_chunks and lengths, kv_storage FUSE_U8_ASYM or
 * FUSE_U4_ASYM, its k, v, k_scale, k_zero, v_scale, v_zero are outputs
 * (layouts as in fuse_chunk_t).  With L = 2^b - 1, a group with minimum mn
 * and maximum mx is stored as q = rint((x - mn) / (mx - mn) * L) (round half
 * to even, in fp64), scale = fp16((mx - mn) / L), zero = fp16(mn); a constant
 * group gets q = 0 and scale 0.  Key groups: (chunk, head, channel) over the
 * chunk's tokens; value groups: (token, head) over d.  Argument errors
 * (mismatched tables, other layouts or storage) are returned before any
 * launch. */
fuse_status_t fuse_kivi_quantize(const fuse_layer_desc_t* desc, const fuse_chunks_t* src,
                                 const fuse_chunks_t* dst, fuse_stream_t stream);

/* ---------------------------------------------------------------------- */
/* Attention without a fused cache: new tokens over the chunk caches as they
 * are stored, and whole packed prompts.                                    */

/* Attention of the last n_new tokens of every request straight over its
 * chunk caches in their storage form (codes of 4 or 8 bits, or layer type;
 * contiguous or paged): what fuse_stitch_rerotate, fuse_recompute_selected's
 * scatter and a causal attention over the fused cache give, without writing
 * that cache.  For request r with its chunks (those whose rows lie in
 * [row0, row0 + N_r)), the new token u (0 <= u < n_new) is its query token
 * j = Qn_r - n_new + u, and with s over the keys that it sees
 *   O[r * n_new + u, h] = softmax_s(q_{u,h} . k_s[h/g] / sqrt(d)) v_s[h/g]:
 *   - every chunk token at a request position not in idx_r:
 *     k = R^{pos} K_i[t], v = V_i[t], dequantised, in fp32 (never rounded to
 *     the layer type);
 *   - the k_r refreshed rows of the selected positions and the query tokens
 *     0 .. j (j included): rows of Ks and Vs, already rotated.
 * R^{pos} and the keys' scales are applied to q (q . R^pos k = R^-pos q . k),
 * so each code is read once and used as it is.
 *   Q, O    [n_req * n_new, Hq, d]  request-major; Q rotated at its positions.
 *   idx     as for fuse_recompute_selected (may be NULL when every k_r is 0).
 *   Ks, Vs  [R_total, Hkv, d] in desc->dtype, request r's rows at [out0,
 *           out0 + k_r + Qn_r): its k_r refreshed context tokens, then its
 *           query tokens (the prompt's query and what was generated since).
 *           out0 may leave room between requests, so that Qn_r can grow.
 * Chunk storage: FUSE_U4_ASYM, FUSE_U8_ASYM or desc->dtype.  Requirements
 * (else FUSE_ERR_INVALID_ARG): 1 <= n_new <= 8 and n_new <= Qn_r; requests
 * in row order and disjoint; chunks sorted by dst_row, not overlapping, each
 * inside one request's context.  A pool of more than 2^31 - 1 token rows is
 * FUSE_ERR_UNSUPPORTED.  A block id outside the pool drops its
 * tokens, a selected index out of range or order is ignored; both are
 * recorded as FUSE_ERR_DEVICE_BOUNDS.  Softmax statistics and sums are fp32;
 * no atomics: equal inputs give equal outputs.  In bf16 layers a weight meets
 * the values in fp16 beside codes (with the value's scale), in two bf16 parts
 * beside rows.  What a row does not see does not reach it, infinities and NaN
 * included (the scales of a chunk whose every token is selected among them); of
 * what it sees, a key of score -infinity has no weight and an infinite value
 * makes its element infinite.  O may not overlap an input.
 * A captured call keeps the tables' sizes of its capture.  The workspace (of
 * fuse_attend_workspace_size, convention as for fuse_workspace_size) is
 * written before it is read. */
#define FUSE_ATTEND_MAX_NEW 8
fuse_status_t fuse_attend_workspace_size(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                                         const fuse_requests_t* reqs, int32_t n_new, size_t* bytes);
fuse_status_t fuse_attend_chunks(const fuse_layer_desc_t* desc, const fuse_chunks_t* chunks,
                                 const fuse_requests_t* reqs, int32_t n_new, const void* Q,
                                 const int32_t* idx, const void* Ks, const void* Vs, void* O,
                                 void* ws, size_t ws_bytes, fuse_stream_t stream);

/* Causal attention of whole prompts packed back to back ([KVBoost] section
 * 3.1, Eq. 2, on every row): request r's rows are [row0, row0 + T_r),
 * T_r = N_r + Qn_r (N_r and Qn_r only add up here; k, sel0, out0 and score0
 * are not used), and row s of it
 *   O[row0 + s, h] = softmax_{j <= s}(q_{s,h} . K[row0 + j, h/g] / sqrt(d)) V[row0 + j, h/g].
 * With one request per chunk it is the attention inside independently
 * computed chunks ([QCFuse] Eq. 3), with one per prompt that of a prompt
 * without reuse.  Q, O: [T_total, Hq, d]; K, V: [T_total, Hkv, d]; Q and K
 * rotated by the caller.  Rows outside every request are neither read nor
 * written, and nothing that a row does not see reaches it, infinities and
 * NaN included; a key of score -infinity has no weight.  Statistics and sums
 * are fp32; in bf16 layers the weights are rounded to bf16 where they meet the
 * values (their sum is that of the unrounded ones).  Requests must be in row
 * order and disjoint (else FUSE_ERR_INVALID_ARG).  O may not overlap Q, K or V.  Needs the workspace
 * of fuse_workspace_size. */
fuse_status_t fuse_attend_prompt(const fuse_layer_desc_t* desc, const fuse_requests_t* reqs,
                                 const void* Q, const void* K, const void* V, void* O, void* ws,
                                 size_t ws_bytes, fuse_stream_t stream);

/* ---------------------------------------------------------------------- */
/* Upkeep of a paged cache.  A pool has n_pool_blocks pages of block_size
 * tokens; sequences name them in block tables (fuse_chunk_t.block_table and
 * len of a FUSE_KV_PAGED chunk table; its other fields are not used here).
 * refs [n_pool_blocks] int32 (device) counts the table entries that name
 * each page; 0 is a free page.  Fork, free and compact keep tables and refs;
 * what has to be copied goes to a move list,
 *   moves [2 + 2 * max_moves] int32 (device): the number of moves, the number
 *   of live pages after the call, then (source page, destination page) pairs,
 * which fuse_pages_copy applies to each layer's pool.  Every table that names
 * pages of the pool has to be in the table given to fuse_pages_compact.
 * Workspace: fuse_pages_workspace_size of the same chunk table (NULL: what
 * fuse_pages_free and fuse_pages_copy need, its header); calls on different
 * streams need their own. */

/* Bytes of workspace for fork and compact on these tables. */
fuse_status_t fuse_pages_workspace_size(const fuse_chunks_t* tables, size_t* bytes);

/* Branch off sequences: dst's table i (device memory that is written,
 * ceil(len / block_size) entries) shares the full pages of src's table i
 * (refs + 1) and gets a page of its own in place of a partly filled last one:
 * the lowest-numbered free pages, in table order, listed in moves.  The same
 * source may appear any number of times; no dst table may overlap another or
 * a source.  src and dst have the same lengths.  max_moves must be at least
 * the number of partly filled last pages (else FUSE_ERR_WORKSPACE).  When a
 * source entry is outside the pool or names a free page, or any page's count
 * is negative (FUSE_ERR_DEVICE_BOUNDS), or too few pages are free
 * (FUSE_ERR_NO_PAGES), nothing changes and the move list is empty. */
fuse_status_t fuse_pages_fork(const fuse_chunks_t* src, const fuse_chunks_t* dst, int32_t* refs,
                              int32_t* moves, int32_t max_moves, void* ws, size_t ws_bytes,
                              fuse_stream_t stream);

/* Drop sequences: every entry of every table gives up one reference.  An
 * entry outside the pool, or past the references that its page has, is
 * recorded as FUSE_ERR_DEVICE_BOUNDS and changes nothing.  The tables
 * themselves are left as they are. */
fuse_status_t fuse_pages_free(const fuse_chunks_t* tables, int32_t* refs, void* ws, size_t ws_bytes,
                              fuse_stream_t stream);

/* Pack the pool: with n live pages, the live pages at ids n and above move,
 * in order, to the free ids below n (as few moves as can be; sources and
 * destinations are disjoint); tables and refs are rewritten.  max_moves must
 * be at least n_pool_blocks / 2 (else FUSE_ERR_WORKSPACE).  An entry outside
 * the pool or naming a free page, or a negative count of any page, is recorded
 * as FUSE_ERR_DEVICE_BOUNDS, and then nothing changes and the move list is
 * empty. */
fuse_status_t fuse_pages_compact(const fuse_chunks_t* tables, int32_t* refs, int32_t* moves,
                                 int32_t max_moves, void* ws, size_t ws_bytes,
                                 fuse_stream_t stream);

/* The pages of one layer: k, v [n_blocks, block_size, Hkv, d] (d / 2 bytes
 * for FUSE_U4_ASYM), v_scale, v_zero [n_blocks, block_size, Hkv] fp16 for
 * coded storage (as the PAGED fields of fuse_chunk_t). */
typedef struct {
  void* k;
  void* v;
  void* v_scale;
  void* v_zero;
} fuse_pool_t;

typedef struct {
  int32_t n_pools;
  int32_t kv_storage;   /* fuse_dtype_t */
  int32_t block_size;
  int32_t reserved;     /* must be 0 */
  int64_t n_blocks;
  const fuse_pool_t* h_pools;   /* host [n_pools] */
} fuse_pools_t;

/* Copy whole pages within every pool: for each pair of the move list, page
 * src to page dst (rows past a sequence's end included).  moves is read on
 * the device, so the list of a fork or compaction enqueued just before
 * applies.  No destination may be another pair's source or destination (the
 * lists of fork and compact never are; otherwise those pages' contents are
 * unspecified).  A count above max_moves copies nothing, a page outside the
 * pool skips its pair; both are recorded as FUSE_ERR_DEVICE_BOUNDS. */
fuse_status_t fuse_pages_copy(const fuse_layer_desc_t* desc, const fuse_pools_t* pools,
                              const int32_t* moves, int32_t max_moves, void* ws, size_t ws_bytes,
                              fuse_stream_t stream);

/* ---------------------------------------------------------------------- */
/* A speculative step over a paged cache: rotate new rows and write them to
 * their pages, attend a tree of drafted tokens, verify the drafts, keep the
 * accepted ones.                                                           */

/* Sequences held in pages, their lengths and tables on the device (written by
 * fuse_cache_keep, or by the caller): nothing of a step needs the host.
 * Sequence s holds lens[s] tokens in the pages tables[s][0 ..]: token t in row
 * t % block_size of page tables[s][t / block_size].  A call brings it the rows
 * rows[s] .. rows[s + 1] - 1 of its row tensors (none is fine), its new tokens
 * 0, 1, ..; new token i belongs in slot lens[s] + i.  Rows in front of rows[0]
 * and from rows[n_seq] on are not written, and what they hold reaches nothing
 * (they may be read, up to n_rows).
 * A contiguous cache is one of large pages.  So is the fused cache of a request
 * where its row0 is a multiple of block_size; requests packed at any row have
 * pages of one token (table entry t: row0 + t).  Pages behind the fused rows
 * take the new tokens.
 * Trees.  parents [n_rows] int32 (device) gives each new token the number,
 * within its sequence, of the one that it follows: a smaller one, or -1 for
 * what follows the held tokens.  NULL: each follows the one before it.
 * The tokens of a table's row and of the pool number less than 2^31 - 256 (else
 * FUSE_ERR_UNSUPPORTED), sequences at most 65535.
 * A sequence whose row starts descend or pass n_rows, that has more than
 * max_new rows, whose length is negative, or whose slots pass the table's row
 * is recorded as FUSE_ERR_DEVICE_BOUNDS and left out (where row starts descend,
 * rows that two sequences claim may be, too).  A parent out of range is
 * recorded and read as -1. */
typedef struct {
  int32_t n_seq;
  int32_t block_size;      /* tokens per page (> 0)                              */
  int32_t max_blocks;      /* entries of a table row (> 0)                       */
  int32_t max_new;         /* rows of a sequence in a call, at most (> 0)        */
  int64_t n_pool_blocks;   /* pages of the pool                                  */
  const int32_t* tables;   /* device [n_seq, max_blocks]                         */
  int32_t* lens;           /* device [n_seq]                                     */
  const int32_t* rows;     /* device [n_seq + 1], ascending                      */
} fuse_seqs_t;

#define FUSE_TREE_MAX_NEW 64   /* new tokens of a sequence in a tree */

/* Workspace of the calls below that say so: its header only. */
#define FUSE_CACHE_WORKSPACE 256

/* Rotary positions of fuse_cache_append.  The first rot_dim channels of a head
 * are rotated (0: all; a multiple of 16), in pairs m = 0 .. rot_dim / 2 - 1:
 *   FUSE_ROPE_HALF         channels m and m + rot_dim / 2
 *   FUSE_ROPE_INTERLEAVED  channels 2m and 2m + 1
 * by position * theta'_m; the rest is copied.  With theta_m = rope_base^(-2m / rot_dim):
 *   FUSE_ROPE_PLAIN   theta' = theta
 *   FUSE_ROPE_LINEAR  theta' = theta / factor
 *   FUSE_ROPE_LLAMA3  theta' = (1 - c) theta / factor + c theta, with
 *                     c = clamp((original_len theta / 2 pi - low) / (high - low), 0, 1)
 *   FUSE_ROPE_YARN    theta' = (1 - r) theta + r theta / factor, with
 *                     r = clamp((m - a) / max(b - a, 0.001), 0, 1),
 *                     a = max(0, floor(t(high))), b = min(rot_dim - 1, ceil(t(low))),
 *                     t(x) = rot_dim ln(original_len / (2 pi x)) / (2 ln rope_base)
 * mscale (1 without one) multiplies the rotated channels.  Angles are reduced
 * exactly (64-bit fractions of a turn), whatever the position. */
typedef enum { FUSE_ROPE_HALF = 0, FUSE_ROPE_INTERLEAVED = 1 } fuse_rope_layout_t;
typedef enum {
  FUSE_ROPE_PLAIN = 0,
  FUSE_ROPE_LINEAR = 1,
  FUSE_ROPE_LLAMA3 = 2,
  FUSE_ROPE_YARN = 3
} fuse_rope_scaling_t;
typedef struct {
  int32_t layout;          /* fuse_rope_layout_t  */
  int32_t rot_dim;
  int32_t scaling;         /* fuse_rope_scaling_t */
  int32_t original_len;
  double factor;           /* >= 1 (LINEAR, LLAMA3, YARN) */
  double low, high;        /* 0 < low < high (LLAMA3, YARN) */
  double mscale;           /* > 0, as a float */
} fuse_rope_t;

/* The rows of fuse_cache_append, in desc->dtype.  Q, K and V may be parts of
 * wider rows (one fused projection): row i starts stride * i elements on, its
 * heads are contiguous.  Strides are multiples of 16 bytes. */
typedef struct {
  const void* Q;           /* [n_rows, Hq, d]; NULL: none                        */
  const void* K;           /* [n_rows, Hkv, d]                                   */
  const void* V;           /* [n_rows, Hkv, d]                                   */
  int64_t q_stride, k_stride, v_stride;
  void* Qr;                /* [n_rows, Hq, d] rotated, contiguous (Q's memory if
                              Q is contiguous); NULL with Q NULL                 */
  void* Kr;                /* [n_rows, Hkv, d] the same for K; may be NULL       */
  void* k_pool;            /* [n_pool_blocks, block_size, Hkv, d]                */
  void* v_pool;
} fuse_append_t;

/* Rotate the new rows ([KVBoost] Eq. 3) and write them to their pages: row i of
 * sequence s has position lens[s] + depth(i), depth the number of its ancestors
 * among the new tokens, and goes to slot lens[s] + i:
 *   Qr = R^pos Q,  k_pool[slot] = R^pos K (also Kr),  v_pool[slot] = V.
 * lens is not changed: fuse_cache_keep (or the caller) raises it.  Rounded once,
 * to desc->dtype; parts that are not rotated are copied bit for bit.  A page
 * outside the pool is recorded as FUSE_ERR_DEVICE_BOUNDS and not written.
 * With parents, max_new is at most FUSE_TREE_MAX_NEW.  Outputs may not overlap
 * inputs, Qr and Kr in place aside.  ws: FUSE_CACHE_WORKSPACE bytes. */
fuse_status_t fuse_cache_append(const fuse_layer_desc_t* desc, const fuse_rope_t* rope,
                                const fuse_seqs_t* seqs, int64_t n_rows, const int32_t* parents,
                                const fuse_append_t* io, void* ws, size_t ws_bytes,
                                fuse_stream_t stream);

/* Attention of the new tokens of every sequence, already in their pages, over
 * the held tokens and, of the new ones, themselves and their ancestors:
 *   O[i, h] = softmax_k(Q[i, h] . k[h/g] / sqrt(d)) v[h/g]
 * over the slots 0 .. lens[s] - 1 and lens[s] + j for j = i and its ancestors.
 * Q (rotated), O: [n_rows, Hq, d]; max_new <= FUSE_TREE_MAX_NEW; one new token
 * a sequence is the ordinary next-token attention of a paged cache, parents
 * NULL a causal run.  Softmax statistics and sums are fp32; in bf16 layers the
 * weights are rounded to bf16 where they meet the values (their sum is that of
 * the unrounded ones).  What a row does not see does not reach it, infinities
 * and NaN included (rows behind a sequence's last slot among it); a key of
 * score -infinity has no weight, and a row for which nothing has weight is zero.
 * (Sums are formed before they are divided, with weights of up to 2^16: values
 * have to stay below 2^80.)  The slots of a page outside the pool are recorded
 * as FUSE_ERR_DEVICE_BOUNDS and count as not there.  No atomics on sums: equal
 * inputs give equal outputs.  O may not overlap an input.
 * The workspace (of fuse_tree_workspace_size, which depends on the shapes and
 * n_seq only, not on lengths) follows the convention of fuse_workspace_size. */
fuse_status_t fuse_tree_workspace_size(const fuse_layer_desc_t* desc, const fuse_seqs_t* seqs,
                                       size_t* bytes);
fuse_status_t fuse_attend_tree(const fuse_layer_desc_t* desc, const fuse_seqs_t* seqs,
                               int64_t n_rows, const int32_t* parents, const void* Q,
                               const void* k_pool, const void* v_pool, void* O, void* ws,
                               size_t ws_bytes, fuse_stream_t stream);

/* Verify drafted tokens against the target's probabilities, with given random
 * numbers.  Sequence s has the nodes rows[s] .. rows[s + 1] - 1: node 0, the
 * last token that stands, and drafts below it (parents; node 0's is -1).
 *   P   [n_rows, vocab] fp32, row i: the target's distribution after node i
 *   Qd  [n_rows, vocab] fp32, row i: the distribution that node i's children
 *       were drawn from, independently; NULL: drafts were chosen, not drawn
 *   u   [n_rows] in [0, 1): of node i's own acceptance; u_next [n_seq]
 * The walk starts at node 0 with r = P[0], S = 1.  The children c of the node
 * where it stands, in order, with token x = tokens[c]: if r(x) > 0 and
 *   u_c S Qd(x) < r(x)        (Qd NULL: u_c S < r(x))
 * it goes on to c, with r = P[c] and S = 1; else
 *   r = max(r - S Qd, 0), S = sum r   (Qd NULL: S = S - r(x), then r(x) = 0).
 * After the last child, next = the lowest x with r(0) + .. + r(x) > u_next sum r
 * (r = P of the node where nothing of r is left).  Kept tokens and the next one
 * are then distributed as the target's, whatever the drafts.
 *   path [n_seq, max_path]  the nodes walked, node 0 first, then -1
 *   count [n_seq]           their number (0 without rows, next then -1)
 *   next [n_seq]
 * 1 <= max_path <= FUSE_TREE_MAX_NEW; a sequence with more rows is recorded as
 * FUSE_ERR_DEVICE_BOUNDS and treated as one without.  Rows of P and Qd are
 * p_stride and q_stride elements apart (where a row of P lies otherwise against
 * 16 bytes than that of Qd, both are read entry by entry: about twice the time
 * on large vocabularies).  Sums keep about 48 bits.  Entries that
 * are negative, infinite or NaN count as 0; they, tokens outside the vocabulary
 * and parents out of range (never accepted) are recorded where they are read.
 * Random numbers below 0 are read as 0, those from 1 on as the last float before
 * 1; NaN as 0 in u_next, and in u it accepts nothing.  ws: FUSE_CACHE_WORKSPACE bytes. */
fuse_status_t fuse_verify_tree(int32_t n_seq, int64_t n_rows, int32_t vocab, const int32_t* rows,
                               const int32_t* parents, const int32_t* tokens, const float* P,
                               int64_t p_stride, const float* Qd, int64_t q_stride, const float* u,
                               const float* u_next, int32_t max_path, int32_t* path,
                               int32_t* count, int32_t* next, void* ws, size_t ws_bytes,
                               fuse_stream_t stream);

/* Keep the rows of a path in every pool and drop the other new ones: for i <
 * count[s], slot lens[s] + i receives what slot lens[s] + path[s][i] held, and
 * then lens[s] += count[s].  pools: F32 or BF16, as fuse_pages_copy's; seqs:
 * as the rows were appended.  No pool is listed twice (FUSE_ERR_INVALID_ARG).
 * A path that does not ascend or names a row that the sequence does not have, or
 * a count outside [0, max_path], is recorded as FUSE_ERR_DEVICE_BOUNDS and leaves
 * the sequence as it is; so does a page outside the pool.  ws: FUSE_CACHE_WORKSPACE bytes. */
fuse_status_t fuse_cache_keep(const fuse_layer_desc_t* desc, const fuse_pools_t* pools,
                              const fuse_seqs_t* seqs, const int32_t* path, int32_t max_path,
                              const int32_t* count, void* ws, size_t ws_bytes,
                              fuse_stream_t stream);

/* Synchronise the stream, read the workspace's error word, clear it, and
 * return it (FUSE_OK if no device-side error was recorded).  If detail is
 * not NULL it receives a code locating the failed check. */
fuse_status_t fuse_check_errors(void* ws, fuse_stream_t stream, uint32_t* detail);

/* Top-k without a workspace (no counterpart on the pages).  Same selection
 * as fuse_select_topk, for callers that cannot allocate device memory when
 * they select: a serving loop that has given all free HBM to its KV-cache
 * pool, or code running where the allocator must not be touched.  The key
 * scratch is a fixed device array inside the library (4 *
 * FUSE_TOPK_NOALLOC_MAX_KEYS + 256 bytes, 2 MiB), held on every GPU that
 * loads the library until the process exits; this call allocates nothing.
 *   - N_total (the largest score0 + N_r) above FUSE_TOPK_NOALLOC_MAX_KEYS is
 *     rejected with FUSE_ERR_WORKSPACE before any launch.
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current); make that first call before
 *     any stream capture.
 *   - All calls share the one array: calls whose work overlaps on the GPU
 *     (different streams, no ordering between them) race and give wrong
 *     indices.  Order them on one stream or with events.
 *   - NaN scores still rank below every number, but this variant does not
 *     report them (fuse_select_topk with a workspace does). */
#define FUSE_TOPK_NOALLOC_MAX_KEYS (1 << 19)
fuse_status_t fuse_select_topk_noalloc(const fuse_requests_t* reqs, const float* score,
                                       int32_t* idx, fuse_stream_t stream);

/* Static selectors: indices generated from the chunk layout alone, no
 * scores (the query-agnostic selectors of the "Token Selection" related-work
 * section of the QCFuse page, and SelectiveRecompute, "Seam Repair" section
 * of the KVBoost page).  A request's context is the concatenation of the
 * chunks whose fused rows lie in [row0, row0 + N_r); a chunk starts at
 * position s = dst_row - row0 of its request.
 *   FUSE_SEL_CHUNK_HEAD: the first n tokens of every chunk, [s, s + min(n, len))
 *     (EPIC's LegoLink rule: the first tokens of a stitched chunk act as
 *     attention sinks; the page gives no count, so n is a parameter).
 *   FUSE_SEL_SEAM_TAIL: the n tokens before every seam, [max(0, p - n), p)
 *     for each p = s of a chunk that is not the request's first (a seam is
 *     where two chunks join; the page's default is n = 16).
 * The selection of a request is the union of its ranges, ascending.
 * Requirements (else FUSE_ERR_INVALID_ARG): host mirrors of both tables;
 * chunks sorted by dst_row and non-overlapping; every chunk with len > 0
 * inside exactly one request's context rows; n >= 0. */
typedef enum { FUSE_SEL_CHUNK_HEAD = 0, FUSE_SEL_SEAM_TAIL = 1 } fuse_static_sel_t;

/* Host only, no launch: k_out[r] = size of request r's selection (host array
 * of n_req entries), to be written into the request table's k before
 * fuse_static_select. */
fuse_status_t fuse_static_select_count(const fuse_requests_t* reqs, const fuse_chunks_t* chunks,
                                       int32_t kind, int32_t n, int32_t* k_out);

/* Enqueues one kernel that writes each request's selection, ascending, to
 * idx[sel0 .. sel0 + k_r) (device array).  reqs->h_req[r].k must equal the
 * count of fuse_static_select_count (else FUSE_ERR_INVALID_ARG).  The
 * indices feed fuse_recompute_selected like those of fuse_select_topk. */
fuse_status_t fuse_static_select(const fuse_requests_t* reqs, const fuse_chunks_t* chunks,
                                 int32_t kind, int32_t n, int32_t* idx, fuse_stream_t stream);

/* Kernel timing trace (no counterpart on the pages; a measurement aid).
 * fuse_trace_begin(n) creates n pairs of CUDA events and, until
 * fuse_trace_end, records one pair around each kernel the library launches,
 * on that launch's stream; launches past n are not recorded.  fuse_trace_end
 * waits for the recorded events and writes up to max_out entries
 * {kernel name (static string), elapsed ms} in launch order, *n_out their
 * count.  Host-side state: one trace at a time per process.  Do not open a
 * trace while a stream is being captured into a CUDA graph. */
typedef struct {
  const char* kernel;
  float ms;
} fuse_trace_entry_t;

fuse_status_t fuse_trace_begin(int32_t max_records);
fuse_status_t fuse_trace_end(fuse_trace_entry_t* out, int32_t max_out, int32_t* n_out);

/* Self-test of the device-side failure detection (no counterpart on the
 * pages; a diagnostic).  Launches one CTA on `stream` whose thread waits,
 * through the same bounded mbarrier wait every pipeline of the library uses,
 * on a barrier that nothing arrives on.  When the wait gives up (after its
 * one-second limit) the kernel records FUSE_ERR_TIMEOUT in the workspace's
 * error word and returns, so the context stays usable: fuse_check_errors then
 * returns FUSE_ERR_TIMEOUT.  ws: a workspace of at least 256 bytes (only its
 * header is used), 256-byte aligned.  No fault, trap or endless wait is
 * involved. */
fuse_status_t fuse_selftest_wait_timeout(void* ws, size_t ws_bytes, fuse_stream_t stream);

/* A static, human-readable name of a status code. */
const char* fuse_status_string(fuse_status_t status);

/* Library version, major * 10000 + minor * 100 + patch. */
int32_t fuse_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FUSEKV_H */
