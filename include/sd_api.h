/*
 * sd_api.h -- C ABI of the top-k sparse decode library for NVIDIA B200 (sm_100a).
 *
 * One decode step over a paged KV cache, for a batch of B requests with one
 * query token each:
 *
 *   1. indexer score  s[b,g,t] = sum_h w[b,g,h] * max(0, sum_d qi[b,g,h,d] * ki[t,g,d])
 *                     for every cached token t < seqlens[b], keys read in place
 *                     from the paged indexer pool through the block table;
 *   2. top-k          per (request, KV head) the min(k, seqlen) tokens of highest
 *                     score, ties to the lower token index, written in ascending
 *                     token order and padded with -1;
 *   3. sparse attn    o[b,h] = sum_j softmax_j(scale * q[b,h] . K_j) V_j over the
 *                     selected rows of KV head g = h / (H/G), gathered from the
 *                     paged K/V pools, followed by a split combine.
 *
 * Where this comes from. The pages describe the DSA decode data flow: an
 * indexer scores the cached tokens, a top-k kernel fills a persistent top-k
 * buffer, and core sparse attention consumes it ("Overlap DSA heuristic
 * prev_topk write-back on the aux stream", Description). Predicted indices are
 * request-local token ids translated to pool rows through the block table, and
 * negative entries are invalid ("Unify sparse attention framework with clean
 * backend interfaces", review notes on DSA global index conversion). The golden
 * reference attends over selected tokens of a logical cache rebuilt from
 * pages ("Add DSA Vanilla sparse attention", Walkthrough). A typed, fixed
 * signature beats a generic keyword carrier ("Compact pseudo-KV/topological
 * sparse attention benchmark evidence", the 0.756x kwargs result). The pages
 * never write the formulas out; the readings taken (ReLU per indexer head,
 * integer head weights, lowest-index ties, ascending order) are stated in the
 * design notes.
 *
 * Conventions for every call
 *   - All array pointers are DEVICE pointers owned by the caller; the library
 *     never allocates, frees or keeps them. Arrays are dense, row-major, with
 *     the shapes given per argument. bf16 arrays are passed as raw uint16 bits.
 *   - Pools are NHD: [num_pages, page_size, kv_heads, dim]. Token t of request
 *     b lives at page block_table[b * max_pages_per_req + t / page_size],
 *     slot t % page_size.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream). Every call only
 *     enqueues work on it: no host synchronisation, no allocation, so a call can
 *     be captured in a CUDA graph. Buffers keep the addresses the caller gives.
 *   - `workspace` is caller-owned device scratch of at least the size that
 *     sd_workspace_size() returns for the same shape (256-byte aligned).
 *   - The library sets each kernel's shared-memory limit once per device and
 *     remembers it. A device reset (cudaDeviceReset) clears such settings:
 *     unload the library (or restart the process) after one.
 *   - Argument errors are found on the host before any launch and returned as
 *     a status; nothing is enqueued then. Errors in device-resident data (a
 *     seqlen beyond the block table, a block-table entry outside the pool, an
 *     index at or past seqlen) cannot be seen on the host: the kernels mask the
 *     offending token (a bad indexer page scores INT32_MIN, a bad attention
 *     row is skipped), clamp the length, and OR a bit into a sticky per-device
 *     error word that sd_get_device_errors() reads.
 *
 * Supported shapes (others return SD_ERR_UNSUPPORTED):
 *   indexer  Di in {32, 64, 128}, 1 <= Hi <= 64, G * Di <= 1024
 *   top-k    1 <= k <= 2048, max_seqlen <= 1 << 20
 *   attn     (Dk, Dv) in {(64, 64), (128, 128), (576, 512)}, H % G == 0,
 *            H / G <= 128; with v_pages == NULL, V is the first Dv columns of
 *            the K row (MLA latent rows, or MQA with V = K)
 */
#ifndef SD_API_H
#define SD_API_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum sd_status {
  SD_OK = 0,
  SD_ERR_INVALID_ARG = 1,   /* null pointer, negative size, inconsistent shape */
  SD_ERR_UNSUPPORTED = 2,   /* a valid shape this build has no kernel for      */
  SD_ERR_WORKSPACE = 3,     /* workspace missing, too small or misaligned      */
  SD_ERR_CUDA = 4           /* a CUDA runtime call failed (see sd_last_cuda_error) */
} sd_status;

/* Bits of the sticky per-device error word (sd_get_device_errors). */
#define SD_DEVERR_SEQLEN 0x1u   /* seqlens[b] < 0, > max_seqlen or > the block table  */
#define SD_DEVERR_PAGE 0x2u     /* a needed block-table entry outside [0, num_pages)  */
#define SD_DEVERR_INDEX 0x4u    /* an attention index >= seqlens[b] (row skipped)     */
#define SD_DEVERR_TIMEOUT 0x8u  /* a bounded on-chip wait ran out (the kernel unwound) */

/* Geometry shared by the indexer pool and the K/V pools of one cache. */
typedef struct sd_paged_desc {
  int32_t num_pages;          /* pages in each pool                           */
  int32_t page_size;          /* tokens per page, >= 1                        */
  int32_t max_pages_per_req;  /* row stride of block_table                    */
  int32_t kv_heads;           /* G: KV heads (1 for MLA latent rows)          */
} sd_paged_desc;

/* Device scratch (bytes) that any of the three calls below needs for this
 * shape: scores (unless the caller passes its own), top-k state and split
 * attention partials. Pure function of its arguments; 0 on invalid input. */
size_t sd_workspace_size(int32_t B, int32_t G, int32_t max_seqlen, int32_t k,
                         int32_t H, int32_t Dv);

/* Steps 1 + 2: indexer scores and per-(request, KV head) top-k.
 *   qi          int8  [B, G, Hi, Di]  indexer queries
 *   w           int32 [B, G, Hi]      indexer head weights
 *   ki_pages    int8  [num_pages, page_size, G, Di]  indexer key pool, 16-byte
 *               aligned (SD_ERR_INVALID_ARG otherwise)
 *   block_table int32 [B, max_pages_per_req]  physical page per logical page
 *   seqlens     int32 [B]             cached tokens per request (incl. current)
 *   max_seqlen  host upper bound of seqlens (sizes grids and scores)
 *   indices     int32 [B, G, k]  OUT  ascending request-local tokens, -1 padded
 *   scores      int32 [B, G, max_seqlen]  OUT, nullable; entries t >= seqlens[b]
 *               are left unwritten. When NULL the scores live in the workspace. */
sd_status sd_indexer_topk(const int8_t* qi, const int32_t* w, const int8_t* ki_pages,
                          const int32_t* block_table, const int32_t* seqlens,
                          sd_paged_desc pd, int32_t B, int32_t Hi, int32_t Di,
                          int32_t max_seqlen, int32_t k, int32_t* indices, int32_t* scores,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Step 3: attention over selected rows, then the split combine.
 *   q        bf16 [B, H, Dk]
 *   k_pages  bf16 [num_pages, page_size, G, Dk]
 *   v_pages  bf16 [num_pages, page_size, G, Dv], or NULL: V = K row[:Dv]
 *   indices  int32 [B, G, k] request-local tokens. Only the first min(k, seqlens[b])
 *            slots of a row are read (a selection has at most seqlen distinct
 *            tokens, so it fits there); entries < 0 in them are skipped
 *   scale    softmax scale applied to q . K
 *   out      bf16 [B, H, Dv] OUT (round to nearest even); zero when nothing is selected
 *   lse      fp32 [B, H] OUT, nullable: natural-log sum of exp(scale * q . K_j),
 *            -inf when nothing is selected */
sd_status sd_sparse_attn(const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages,
                         const int32_t* block_table, const int32_t* seqlens,
                         const int32_t* indices, sd_paged_desc pd, int32_t B, int32_t H,
                         int32_t Dk, int32_t Dv, int32_t k, float scale, uint16_t* out,
                         float* lse, void* workspace, size_t workspace_bytes, void* stream);

/* TriAttention-style decode-time eviction of one layer ("Add TriAttention
 * KV-cache compression method", Summary and Key Design Decisions): score the
 * evictable region [n_sink, L_b - n_recent) of every request with calibrated
 * per-head queries, keep the `budget` best tokens, and compact the kept K/V
 * rows in place to the front of the request's pages.
 *   q_cal       bf16 [H, D]: one calibrated query per query head (head h reads
 *               KV head h * G / H), in the cache's precision
 *   k_pages     bf16 [num_pages, P, G, D], compacted in place; 16-byte aligned
 *   v_pages     bf16 [num_pages, P, G, D] compacted the same way, or NULL;
 *               16-byte aligned
 *   mode        SD_TRI_UNION: one selection per request (all KV heads move
 *               together); SD_TRI_PER_HEAD (or SD_TRI_PER_LAYER_PER_HEAD):
 *               one per (request, KV head)
 *   new_seqlens int32 [B] out: n_sink + budget + n_recent, or L_b when the
 *               evictable region holds at most `budget` tokens (nothing moves)
 * Score of evictable position p under query head h: z = q_cal[h] . K, summed
 * in fp32 (each bf16 x bf16 product exact; one fused multiply-add per d, so
 * equal inputs give equal scores), shifted by the head's maximum over the
 * region; a KV head's score is the maximum over its query heads, the union
 * score the maximum over KV heads. The `budget` largest are kept (ties to the
 * lower position), followed by the recent tail. The kept set is a top-budget
 * set of the exact scores up to the fp32 rounding of the sums. Pages past the new
 * lengths are free for the caller to release; the block table is unchanged. If
 * the pools are an sd_kv_cache's, its k_bounds are stale afterwards (see there).
 * max_seqlen is a host upper bound of seqlens (it sizes the workspace);
 * larger lengths are clamped and flag SD_DEVERR_SEQLEN.
 * Limits: D in {64, 128}; H / G in {1, 2, 4, 8}; H <= 256;
 * 1 <= budget <= 2048; B * G <= 65535; the bytes one token moves (union:
 * G * D * 2, per-head: D * 2; twice that with V) at most 32768.
 * block_table, seqlens and new_seqlens may be NULL when B = 0.
 * Workspace: sd_tri_workspace_size(); the caller owns every buffer.
 * Errors: SD_ERR_INVALID_ARG / SD_ERR_UNSUPPORTED / SD_ERR_WORKSPACE before
 * any launch. A block-table entry outside the pool inside a request sets
 * SD_DEVERR_PAGE and that row is skipped (the request's result is then
 * unspecified, the pools outside its pages untouched). The compaction's
 * units wait on one another with bounded waits; one that runs out sets
 * SD_DEVERR_TIMEOUT and skips its writes. */
#define SD_TRI_UNION 0
#define SD_TRI_PER_HEAD 1
#define SD_TRI_PER_LAYER_PER_HEAD 2 /* with one layer, the same as SD_TRI_PER_HEAD */
size_t sd_tri_workspace_size(int32_t B, int32_t G, int32_t H, int32_t D, int32_t max_seqlen, int32_t n_sink,
                             int32_t n_recent, int32_t budget, int32_t mode, int32_t has_v);
sd_status sd_tri_compact(const uint16_t* q_cal, uint16_t* k_pages, uint16_t* v_pages, const int32_t* block_table,
                         const int32_t* seqlens, sd_paged_desc pd, int32_t B, int32_t H, int32_t D, int32_t max_seqlen,
                         int32_t n_sink, int32_t n_recent, int32_t budget, int32_t mode, int32_t* new_seqlens,
                         void* workspace, size_t workspace_bytes, void* stream);

/* The same over n_layers layers that share the block table and lengths
 * ("Add TriAttention KV-cache compression method", Summary: union, per_head
 * and per_layer_perhead eviction modes). q_cal, k_pages and v_pages are HOST
 * arrays of n_layers device pointers (v_pages may be NULL: no V pools).
 *   SD_TRI_UNION              one selection per request for every layer and
 *                             head: score = max over layers and heads
 *   SD_TRI_PER_HEAD           one selection per (request, KV head) for every
 *                             layer: score = max over layers and that KV
 *                             head's query heads
 *   SD_TRI_PER_LAYER_PER_HEAD an independent per-head selection in each layer
 * (each head's logits shifted by that layer's and head's maximum, as above).
 * Every layer is compacted; new_seqlens holds the common new lengths.
 * Workspace: sd_tri_layers_workspace_size(). Limits and errors as above. */
size_t sd_tri_layers_workspace_size(int32_t n_layers, int32_t B, int32_t G, int32_t H, int32_t D, int32_t max_seqlen,
                                    int32_t n_sink, int32_t n_recent, int32_t budget, int32_t mode, int32_t has_v);
sd_status sd_tri_compact_layers(const uint16_t* const* q_cal, uint16_t* const* k_pages, uint16_t* const* v_pages,
                                int32_t n_layers, const int32_t* block_table, const int32_t* seqlens, sd_paged_desc pd,
                                int32_t B, int32_t H, int32_t D, int32_t max_seqlen, int32_t n_sink, int32_t n_recent,
                                int32_t budget, int32_t mode, int32_t* new_seqlens, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Steps 1 + 2, and the whole decode step, with the previous step's selection
 * as a hint: the "heuristic_prev_topk" feedback of "Overlap DSA heuristic
 * prev_topk write-back on the aux stream" (Description: each decode step's
 * top-k is the next step's pre_idx hint).
 *   hint  int32 [B, G, k] request-local tokens (-1 and tokens >= seqlen are
 *         ignored), typically the previous call's `indices`; NULL = no hint.
 *         It must not be the same buffer as `indices`.
 * The result is identical to the unhinted call for any hint. A good hint (the
 * previous selection of a slowly changing query) narrows the radix passes of
 * the top-k to the range between the hint's lowest current score and the best
 * score outside it; an exact hint needs no radix pass at all. The write-back
 * of the pages (a copy into the hint buffer) is not needed: alternate two
 * `indices` buffers between steps and pass the other as the hint. Other
 * arguments and errors as for sd_indexer_topk / sd_decode_step. */
sd_status sd_indexer_topk_hinted(const int8_t* qi, const int32_t* w, const int8_t* ki_pages,
                                 const int32_t* block_table, const int32_t* seqlens, sd_paged_desc pd, int32_t B,
                                 int32_t Hi, int32_t Di, int32_t max_seqlen, int32_t k, const int32_t* hint,
                                 int32_t* indices, int32_t* scores, void* workspace, size_t workspace_bytes,
                                 void* stream);
sd_status sd_decode_step_hinted(const int8_t* qi, const int32_t* w, const int8_t* ki_pages, const uint16_t* q,
                                const uint16_t* k_pages, const uint16_t* v_pages, const int32_t* block_table,
                                const int32_t* seqlens, sd_paged_desc pd, int32_t B, int32_t Hi, int32_t Di,
                                int32_t H, int32_t Dk, int32_t Dv, int32_t max_seqlen, int32_t k, float scale,
                                const int32_t* hint, int32_t* indices, int32_t* scores, uint16_t* out, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Steps 3 + 4 for n_layers layers that share one selection: the
 * shared-indexer decode of "Overlap DSA heuristic prev_topk write-back on the
 * aux stream" (Description: layers without their own indexer reuse the top-k
 * buffer) and of "Add DSA Vanilla sparse attention" (the persistent index
 * buffer read by every layer).
 *   q        bf16 [n_layers, B, H, Dk], layer-major
 *   k_pages  HOST array of n_layers device pointers, each a latent / key pool
 *            laid out as for sd_sparse_attn (all with the geometry `pd`)
 *   v_pages  HOST array of n_layers value pools, or NULL (V inside K)
 *   block_table, seqlens, indices: one set, shared by every layer
 *   out      bf16 [n_layers, B, H, Dv]; lse fp32 [n_layers, B, H] or NULL
 * With MLA rows (G = 1, H = 128, Dk = 576, Dv = 512, V inside K), up to 16
 * layers run in one launch, so the selections are resolved to pool rows once
 * per group of layers and small batches fill the GPU; other shapes run layer
 * after layer. Workspace: sd_attn_layers_workspace_size(). Errors as for
 * sd_sparse_attn; SD_ERR_INVALID_ARG also for n_layers < 1 or a NULL pool. */
size_t sd_attn_layers_workspace_size(int32_t n_layers, int32_t B, int32_t G, int32_t k, int32_t H, int32_t Dv);
sd_status sd_sparse_attn_layers(const uint16_t* q, const uint16_t* const* k_pages, const uint16_t* const* v_pages,
                                int32_t n_layers, const int32_t* block_table, const int32_t* seqlens,
                                const int32_t* indices, sd_paged_desc pd, int32_t B, int32_t H, int32_t Dk,
                                int32_t Dv, int32_t k, float scale, uint16_t* out, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Steps 3 + 4 with the selection given in the packed forms of the unified
 * sparse runtime ("Unify sparse attention framework with clean backend
 * interfaces", runtime parameters sparse_attn_offsets and
 * sparse_attn_indices_block_size):
 *   indices     int32, all rows' entries packed (may be NULL if every row is
 *               empty); row r = b * G + g owns indices[offsets[r] ..
 *               offsets[r + 1]).
 *   offsets     int32 [B * G + 1], non-decreasing.
 *   block_size  0 or 1: an entry is a token; bs > 1: entry e selects tokens
 *               e*bs .. e*bs + bs - 1.
 *   max_selected  1 .. 2048: the most tokens any row keeps.
 * Row r attends over the valid tokens of its expansion, in list order: entries
 * < 0 are skipped, tokens at or past seqlens[b] are dropped, and only the
 * first min(max_selected, seqlens[b]) are kept. An entry whose whole block is
 * past the seqlen, decreasing offsets, or more valid tokens than kept set
 * SD_DEVERR_INDEX. Duplicates are attended as listed. Other arguments,
 * outputs and errors as for sd_sparse_attn. Workspace:
 * sd_csr_workspace_size(). */
size_t sd_csr_workspace_size(int32_t B, int32_t G, int32_t max_selected, int32_t H, int32_t Dv);
sd_status sd_sparse_attn_csr(const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages,
                             const int32_t* block_table, const int32_t* seqlens, const int32_t* indices,
                             const int32_t* offsets, int32_t block_size, int32_t max_selected, sd_paged_desc pd,
                             int32_t B, int32_t H, int32_t Dk, int32_t Dv, float scale, uint16_t* out, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Steps 1 + 2 + 3 in one call on one stream (arguments as above). */
sd_status sd_decode_step(const int8_t* qi, const int32_t* w, const int8_t* ki_pages,
                         const uint16_t* q, const uint16_t* k_pages, const uint16_t* v_pages,
                         const int32_t* block_table, const int32_t* seqlens, sd_paged_desc pd,
                         int32_t B, int32_t Hi, int32_t Di, int32_t H, int32_t Dk, int32_t Dv,
                         int32_t max_seqlen, int32_t k, float scale, int32_t* indices,
                         int32_t* scores, uint16_t* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Steps 1 + 2 without any workspace (the pages have no counterpart; this is a
 * deployment convenience). It is sd_indexer_topk for callers that cannot
 * allocate device memory: a plugin that runs inside a host application which
 * owns every device allocation, or a serving loop that must not allocate once
 * it has started. Such callers cannot provide a scores workspace. Here the
 * scores live in a scratch array inside the library's device image:
 * SD_NOALLOC_MAX_SCORES int32 values (16 MiB). It is resident on every device
 * where the library's device code is loaded, whichever entry point loaded
 * it, from then until the context is destroyed.
 *   Arguments, outputs and errors are as for sd_indexer_topk. There is no
 *   scores output. The call returns SD_ERR_WORKSPACE, with nothing enqueued,
 *   when B * G * max_seqlen > SD_NOALLOC_MAX_SCORES.
 *   A call that is not being captured looks up the device's scratch address
 *   (a runtime query, not an allocation) and remembers it; a call under
 *   stream capture uses the remembered address. So make one call on a device
 *   before capturing any, and again after a device reset or anything else
 *   that destroys the primary context (that reloads the library's device
 *   image at another address): a captured graph keeps the address it was
 *   captured with and must be captured anew after such a reset. A first call
 *   on a device made under capture returns SD_ERR_INVALID_ARG.
 *   Every call on a device shares the one scratch array. Calls whose work
 *   overlaps on the GPU (other streams, other threads) race on it and give
 *   undefined results: serialise them. The array keeps the last call's scores,
 *   and that is harmless, because every score a call reads it has written
 *   first. The call never allocates or frees device memory. */
#define SD_NOALLOC_MAX_SCORES (4u << 20)
sd_status sd_indexer_topk_noalloc(const int8_t* qi, const int32_t* w, const int8_t* ki_pages,
                                  const int32_t* block_table, const int32_t* seqlens,
                                  sd_paged_desc pd, int32_t B, int32_t Hi, int32_t Di,
                                  int32_t max_seqlen, int32_t k, int32_t* indices, void* stream);

/* ---------------------------------------------------------------------------
 * A blocked cache: one layer's paged K and V, [num_pages, page_size, kv_heads,
 * D] each, with a page cut into blocks of `block_tokens` slots (block_tokens
 * divides page_size). kv_type is the pools' element type. An 8-bit pool has
 * one fp32 scale per (block, KV head): the value of a code is code * scale.
 * k_bounds holds the smallest and the largest key of every block, KV head and
 * dim, for the selection of blocks; it may be NULL where nothing is selected.
 * Its entries, like the scales, stand for the tokens that the block holds; the
 * keys are those before coding, as bf16. What moves or overwrites K rows other than
 * sd_kv_store leaves the bounds behind: after sd_tri_compact on bf16 pools
 * they are rebuilt by sd_kv_load of all kept tokens and sd_kv_store of those
 * rows as they are (no q, no weights, rot_dim 0).
 * D in {64, 128}, block_tokens <= 128, num_pages * page_size < 2^31 and
 * max_pages_per_req * page_size < 2^30 (SD_ERR_UNSUPPORTED otherwise);
 * block_tokens divides page_size, pools and bounds 16-byte aligned
 * (SD_ERR_INVALID_ARG otherwise). (No counterpart on the pages: they read
 * caches that a serving stack has written.) */
typedef enum sd_kv_type { SD_KV_BF16 = 0, SD_KV_INT8 = 1, SD_KV_E4M3 = 2 } sd_kv_type;

typedef struct sd_kv_cache {
  void* k_pages;      /* [num_pages, page_size, G, D] of kv_type                     */
  void* v_pages;      /* the same                                                    */
  float* k_scales;    /* [num_pages, page_size / block_tokens, G]; 8-bit pools only  */
  float* v_scales;    /* the same                                                    */
  uint16_t* k_bounds; /* bf16 [num_pages, page_size / block_tokens, G, 2, D], or NULL */
  int32_t kv_type;    /* sd_kv_type                                                  */
  int32_t block_tokens;
  int32_t D;
} sd_kv_cache;

/* Norm, rotation and store of new tokens, one launch. The new tokens of request b
 * are rows tok_start[b] .. tok_start[b + 1] - 1 of q, k and v; they become the
 * last positions of the request, seqlens[b] - n .. seqlens[b] - 1 (seqlens
 * counts them). One row per request is a decode step; more are a prompt or a
 * chunk of one. A request may have none.
 *   q, k, v     bf16 rows [n_tokens][H or G heads][D], heads dense, rows
 *               q_stride, k_stride, v_stride elements apart (a packed q, k, v
 *               projection is read in place); 8-byte aligned, strides
 *               multiples of 4. q may be NULL (only K and V are stored)
 *   tok_start   int32 [B + 1], ascending from 0; what rows at or behind
 *               tok_start[B] hold has no effect, and their q_out rows stay as they were
 *   positions   int32 [n_tokens]: the position each row is rotated to, or NULL:
 *               its position in the cache
 *   q_weight, k_weight  bf16 [D] or NULL (no norm): x * rsqrt(mean(x^2) + eps) * weight
 *               over each head
 *   inv_freq    fp32 [rot_dim / 2]: angle of pair i = position * inv_freq[i].
 *               The first rot_dim dims rotate (a multiple of 8, at most D; 0:
 *               none, inv_freq may be NULL), in pairs (i, i + rot_dim / 2), or
 *               (2i, 2i + 1) with interleaved != 0
 *   q_out       bf16 [n_tokens, H, D], 8-byte aligned; may be q where q is dense
 * Arithmetic is fp32; angles are 64-bit fractions of a turn, as exact as fp64
 * products (2^-24 turns at position 2^30). q_out and bf16 pools are rounded once. In
 * an 8-bit pool the scale of a (block, KV head) is
 *   max(amax(new rows) / qmax, the scale it had if it holds earlier tokens, 2^-100)
 * (qmax 127 or 448), codes are round(y / scale) of the fp32 quotient, ties to
 * even, and earlier codes of a block whose scale grew are coded anew,
 * round(code * (old / new)). NaN is stored as
 * code 0 and an infinity as the largest code; neither enters the scale.
 * k_bounds of a block are those of its tokens' bf16 keys. Pool rows, scales and bounds
 * of other blocks are not touched; two requests must not share a block that
 * either writes. A bad block-table entry flags SD_DEVERR_PAGE and that
 * block's rows are not stored; more rows than seqlens[b] flags
 * SD_DEVERR_INDEX and the rows before position 0 are not stored. */
sd_status sd_kv_store(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_stride, int64_t k_stride,
                      int64_t v_stride, const int32_t* tok_start, const int32_t* positions,
                      const int32_t* block_table, const int32_t* seqlens, sd_paged_desc pd, sd_kv_cache kv, int32_t B,
                      int32_t n_tokens, int32_t H, const uint16_t* q_weight, const uint16_t* k_weight, float eps,
                      const float* inv_freq, int32_t rot_dim, int32_t interleaved, uint16_t* q_out, void* stream);

/* Reads the tokens that sd_kv_store with the same tok_start and seqlens stores
 * back as bf16 rows (for example the cached prefix of a prompt, for an
 * attention over bf16 rows): the last n tokens of every request.
 *   k_out, v_out  bf16 [n_tokens, G, D], 16-byte aligned: code * scale, rounded once.
 * Rows at or behind tok_start[B] stay as they were; a token whose page is bad
 * or whose position is negative reads as zeros and is flagged. */
sd_status sd_kv_load(sd_kv_cache kv, const int32_t* tok_start, const int32_t* block_table, const int32_t* seqlens,
                     sd_paged_desc pd, int32_t B, int32_t n_tokens, uint16_t* k_out, uint16_t* v_out, void* stream);

/* Decode attention over an 8-bit blocked cache, one query per request:
 *   z_j = scale * sk_j * (q . k_j), out = sum_j softmax_j(z) * sv_j * v_j
 * over every cached token (indices NULL), or over listed blocks.
 *   q        bf16 [B, H, D], 16-byte aligned
 *   indices  int32 [B, G, n_list]: entry e selects the tokens e * index_block ..
 *            of the request (1: tokens, as sd_indexer_topk writes them; the
 *            blocks of sd_block_topk: its block_tokens). Only the first
 *            min(n_list, ceil(seqlen / index_block)) entries of a row are read; entries < 0 are
 *            skipped, one that starts at or past the seqlen is skipped and
 *            flags SD_DEVERR_INDEX, tokens past the seqlen are dropped,
 *            duplicates are attended as listed
 *   out      bf16 [B, H, D], 8-byte aligned; zero where nothing is attended
 *   lse      fp32 [B, H] or NULL: ln sum exp z, -inf where nothing is attended
 * n_list >= 1 with a list. H % G == 0, H / G <= 128, n_list * index_block <
 * 2^30, fewer than 2^36 tokens (of whole listed blocks) over all requests,
 * pools below 64 GiB. Scales must be finite and not negative (a V scale below
 * 2^-100 counts as 2^-100). A token on a bad page is skipped and flags
 * SD_DEVERR_PAGE. Slots behind a request's last token may hold anything.
 * Logits and sums are fp32, of queries rounded to 2^-22 (int8, H / G <= 8) or
 * 2^-27 of their head's largest entry. Softmax weights, relative to the
 * largest, are fixed point of 32 bits (int8, H / G <= 4) or 24 (int8, H / G
 * <= 8; what is cut is made up for over neighbouring tokens); of their own
 * bits they keep 22 (e4m3, H / G <= 8) or 11 (H / G > 8).
 * kv_type SD_KV_BF16 returns SD_ERR_UNSUPPORTED (sd_sparse_attn reads bf16 pools).
 * Workspace: sd_kv_attn_workspace_size(). */
size_t sd_kv_attn_workspace_size(int32_t B, int32_t G, int32_t H, int32_t D);
sd_status sd_kv_attn(const uint16_t* q, sd_kv_cache kv, const int32_t* block_table, const int32_t* seqlens,
                     const int32_t* indices, int32_t n_list, int32_t index_block, sd_paged_desc pd, int32_t B,
                     int32_t H, float scale, uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                     void* stream);

/* Selection of blocks by a bound on their scores (any kv_type; kv.k_bounds is
 * read, the pools are not): block c of KV head g scores
 *   max over the group's query heads of sum_d max(q_d * lo_d, q_d * hi_d)
 * summed in fp64 and rounded to fp32: at least the largest q . k of the block's
 * keys as they were before coding. (The coded keys of an 8-bit pool may lie outside
 * the bounds by what coding them cost: half a scale in int8, 2^-4 of the
 * value in e4m3, as much again each time the block's scale grew.) A head
 * whose sum is not a number is left out; the bounds are finite.
 *   q        bf16 [B, H, D], 8-byte aligned
 *   indices  int32 [B, G, n_select]  OUT: the first n_first and the last n_last
 *            blocks of the request and the best others, min(n_select, number
 *            of blocks) together, ties to the lower block; ascending, -1 padded
 * 1 <= n_select <= 2048, n_first + n_last <= n_select, max_seqlen <= 2^20 *
 * block_tokens, B * G <= 65535, H / G <= 128. A block on a bad page scores -inf and
 * flags SD_DEVERR_PAGE. max_seqlen is a host upper bound of seqlens.
 * The indices fit sd_kv_attn with index_block = block_tokens, and, on bf16
 * pools, sd_sparse_attn_csr with offsets r * n_select and block_size =
 * block_tokens, while n_select * block_tokens is within its limit of a row.
 * Workspace: sd_block_topk_workspace_size(). */
size_t sd_block_topk_workspace_size(int32_t B, int32_t G, int32_t max_seqlen, int32_t block_tokens);
sd_status sd_block_topk(const uint16_t* q, sd_kv_cache kv, const int32_t* block_table, const int32_t* seqlens,
                        sd_paged_desc pd, int32_t B, int32_t H, int32_t max_seqlen, int32_t n_select, int32_t n_first,
                        int32_t n_last, int32_t* indices, void* workspace, size_t workspace_bytes, void* stream);

/* sd_block_topk and sd_kv_attn over the blocks it selects, in one call
 * (arguments and errors as above). Workspace: sd_kv_block_step_workspace_size(). */
size_t sd_kv_block_step_workspace_size(int32_t B, int32_t G, int32_t H, int32_t D, int32_t max_seqlen,
                                       int32_t block_tokens);
sd_status sd_kv_block_step(const uint16_t* q, sd_kv_cache kv, const int32_t* block_table, const int32_t* seqlens,
                           sd_paged_desc pd, int32_t B, int32_t H, int32_t max_seqlen, int32_t n_select,
                           int32_t n_first, int32_t n_last, float scale, int32_t* indices, uint16_t* out, float* lse,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Stage timing for monitoring and benchmarks (no counterpart on the pages).
 * `events` points to 2 * n cudaEvent_t handles created by the caller; while
 * set, every call of this thread records events[2*i] just before and
 * events[2*i+1] just after stage i on the call's stream, for the stages
 * 0 = indexer scores, 1 = top-k, 2 = split attention, 3 = combine (a stage
 * a call does not run records nothing). n = 0 or events = NULL switches it
 * off. The handles must outlive their use; the library does not own them. */
sd_status sd_set_stage_events(void* const* events, int32_t n);

/* Test hook for the failure path of bounded waits (no counterpart on the
 * pages). The eviction compaction's units wait on one another through flags
 * in global memory (sd_tri_compact); each wait gives up after a bounded number
 * of polls, sets SD_DEVERR_TIMEOUT and skips that unit's writes, so a wait
 * that never ends cannot hang the GPU. This sets that number for compactions
 * launched afterwards by any thread of the process (it is a launch argument,
 * so a captured graph keeps the value it was captured with): polls < 0
 * restores the default of 2^22, 0 makes every such wait give up at once (the
 * compaction then leaves the pools in an unspecified state and flags the
 * timeout). Values above 2^22 return SD_ERR_INVALID_ARG. No other wait of
 * the library is affected. Nothing is enqueued; no CUDA call is made. */
sd_status sd_set_wait_limit(int32_t polls);

/* Reads (and with clear != 0 resets) the sticky device error word of the
 * current device. Synchronises the device: for tests and debugging only. */
sd_status sd_get_device_errors(uint32_t* bits, int32_t clear);

/* Human-readable name of a status. Never NULL. */
const char* sd_status_str(sd_status status);

/* The cudaError_t of the last failing CUDA call in this thread (0 if none). */
int32_t sd_last_cuda_error(void);

/* Number of kernel launches the last successful call enqueued (per thread). */
int32_t sd_last_launch_count(void);

/* Library ABI version, (major << 16) | minor. */
int32_t sd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SD_API_H */
