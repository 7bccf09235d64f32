/*
 * medusa_tree.h -- C ABI of the Medusa tree-verification library (sm_103a).
 *
 * One verify step of Medusa speculative decoding, for every sequence of a
 * batch, in three calls on one CUDA stream:
 *
 *   mt_tree_attn_paged    the T candidate tokens of the sequence's speculation
 *                         tree attend, in one pass, to the sequence's paged KV
 *                         cache plus their own tree ancestors (the "tree mask"),
 *                         with RoPE applied at position prefix_len + depth;
 *   mt_tree_accept_greedy per-node vocab argmax of the target logits and the
 *                         longest root path whose tokens match their parent's
 *                         argmax;
 *   mt_kv_commit          the accepted nodes' K/V move into the sequence's next
 *                         cache slots, the sequence length grows and the tree
 *                         scratch pages past the new length are released;
 *
 * or in two, with mt_tree_accept_commit doing the last two in one launch.
 * mt_tree_accept_typical replaces greedy acceptance by typical acceptance
 * (a tempered-probability threshold), and mt_tree_candidates builds the tree's
 * tokens from the Medusa heads before the step.  Around the step:
 * mt_qk_norm_rope normalises and rotates queries and keys, mt_kv_append_paged
 * fills the cache, mt_tree_attn_paged_block8 attends over an 8-bit cache with
 * block scales, and mt_sample_tokens draws a token.
 *
 * What the pages fix, per call:
 *  - vLLM issue 1171 "[Discussion] Will vLLM consider using Speculative
 *    Sampling to accelerating LLM decoding?": several new tokens attend to an
 *    existing paged KV cache (comment by zhaoyang-star); the Medusa tree mask
 *    is applied inside the cached-KV attention; block tables are updated when a
 *    candidate is accepted and the other blocks released; the step returns a
 *    list of tokens (comment by void-main listing the needed changes); with
 *    several query tokens per sequence the products belong on tensor cores
 *    (void-main on PagedFlashAttention).
 *  - TensorRT-LLM issue 1946 "How to use Medusa to support non llama models?",
 *    answer by rakib-hasan: a position-offset tensor lets RoPE rotate each
 *    Medusa token at its own position.
 *  - lmdeploy PR 1231 "[WIP] support Medusa": greedy acceptance at LM-head
 *    temperature 0 over a 64-choice tree; a tree-mask kernel in the
 *    Flash-Decoding style (split keys, merge partial softmaxes).
 *  - mlc-llm issue 2319 "[Feature Request] Medusa support": tree attention and
 *    the KV cache update are the two hard parts.
 *
 * Conventions (all calls):
 *  - Every tensor is caller-owned device memory, dense, in the layouts given
 *    below, 16-byte aligned.  The library allocates device memory only in
 *    mt_rope_create.
 *  - Calls are asynchronous on `stream` and never synchronise, except
 *    mt_read_status and mt_rope_create.
 *  - Errors the host can see (null pointers, unsupported dtype / head_dim /
 *    tree size, misalignment, a workspace that is too small) return a negative
 *    mt_status before anything is launched.  Errors only the device can see
 *    (malformed trees, page ids out of range, block tables shorter than
 *    prefix + T slots, a bounded wait that gave up) are recorded in a status
 *    word inside the workspace and read with mt_read_status; the outputs of
 *    an affected sequence are then unspecified, and nothing outside the
 *    caller's buffers is touched.  No kernel traps or asserts.
 *  - Node order: node 0 is the root (parent -1, depth 0): the token chosen by
 *    the previous step, not yet in the cache.  Every other node i has
 *    0 <= parent[i] < i and depth[i] = depth[parent[i]] + 1.  T <= 64.
 *  - Paged cache layout: k_cache and v_cache are [num_pages][Hkv][P][D] in the
 *    act dtype; logical slot s of sequence b is row s % P of page
 *    block_tables[b][s / P].  block_tables is int32 [B][max_blocks_per_seq]
 *    (unused entries may hold -1); seq_lens is int32 [B], the committed prefix
 *    length L_b.  The table must cover slots 0 .. L_b + T - 1: slots
 *    L_b .. L_b + T - 1 are the tree's scratch region.
 */
#ifndef MEDUSA_TREE_H_
#define MEDUSA_TREE_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MT_OK = 0,
  MT_ERR_INVALID_ARG = -1,  /* null pointer, bad size, misaligned, workspace too small */
  MT_ERR_UNSUPPORTED = -2,  /* dtype / head_dim / page size / tree size not supported */
  MT_ERR_TREE = -3,         /* (device) parents or depths violate the node-order rule */
  MT_ERR_PAGES = -4,        /* (device) page id out of range or block table too short */
  MT_ERR_CUDA = -5,         /* a CUDA runtime call failed */
  MT_ERR_TIMEOUT = -6,      /* (device) a bounded pipeline wait gave up */
  MT_ERR_POSITION = -7      /* (device) a position at or past the RoPE table's end */
} mt_status;

/* MT_E4M3 is a cache element type only (see mt_attn_desc.cache_dtype). */
typedef enum { MT_F32 = 0, MT_F16 = 1, MT_BF16 = 2, MT_E4M3 = 3 } mt_dtype;

/* Kernel choice for mt_tree_attn_paged.  AUTO: tensor cores (tcgen05, TMEM,
 * TMA) for fp16/bf16, the SIMT kernel for fp32.  SIMT: the CUDA-core kernel for
 * every dtype (a second, independent implementation used by the tests). */
typedef enum { MT_KERNEL_AUTO = 0, MT_KERNEL_SIMT = 1, MT_KERNEL_TC = 2 } mt_kernel;

typedef struct {
  int batch;               /* B >= 1 */
  int tree_size;           /* T, 1..64 */
  int num_q_heads;         /* Hq, a multiple of Hkv */
  int num_kv_heads;        /* Hkv */
  int head_dim;            /* D: 64 or 128 */
  int page_size;           /* P: 16 */
  int max_blocks_per_seq;  /* columns of block_tables */
  int num_pages;           /* pages in the cache pool */
  int num_splits;          /* 0: balanced schedule over the whole batch (each
                              persistent CTA takes an equal share of all key
                              tiles); n > 0: every (sequence, KV head) is split
                              into n key chunks merged by a log-sum-exp pass */
  mt_dtype dtype;          /* q, k_new, v_new, out, and the caches unless cache_dtype says
                              otherwise */
  float sm_scale;          /* softmax scale; 0 means 1/sqrt(D) */
  int kernel;              /* an mt_kernel value */
  /* FP8 KV cache (a reading: the pages this library follows define none).
   * cache_dtype 0: the caches hold dtype.  MT_E4M3: they hold OCP FP8 E4M3
   * codes (no infinities; largest finite 448) of value / scale, one scale for
   * K and one for V, and every cached element stands for decode(code) *
   * scale, the tree's own K/V included: mt_tree_attn_paged writes the code of
   * (act-rounded rotated key or raw value) / scale, divided in fp32 and
   * rounded to nearest even with saturation to +-448, and reads every visible
   * slot back through the scale.  Runs on either kernel: the tensor-core
   * kernel (fp16/bf16 dtype) loads the codes with TMA, converts them exactly
   * to the act dtype in shared memory, and applies k_scale with the softmax
   * scale and v_scale to the output; MT_KERNEL_AUTO picks it as for a 16-bit
   * cache.  mt_kv_commit and mt_tree_accept_commit move the 1-byte elements.
   * k_scale, v_scale: positive and finite for MT_E4M3, ignored otherwise. */
  int cache_dtype;
  float k_scale;
  float v_scale;
} mt_attn_desc;

/* ---- RoPE table ----------------------------------------------------------
 * Library-owned fp32 cos/sin table [max_pos][D/2] on the current device, built
 * on the host in double precision (NeoX / LLaMA half-split form):
 *   inv_freq_j = pow(base, -(2j)/D), theta = pos * inv_freq_j (IEEE double),
 *   stored values (float)cos(theta), (float)sin(theta).
 * The rotation of a head vector x at position pos, for j < D/2, in fp32 with
 * each product and sum rounded separately (no fused multiply-add):
 *   x'[j] = x[j]*c - x[j+D/2]*s,   x'[j+D/2] = x[j+D/2]*c + x[j]*s,
 * then rounded to nearest-even in the act dtype.  Tree token i of sequence b is
 * rotated at pos = seq_lens[b] + tree_depths[b][i] (the Medusa position offset,
 * TensorRT-LLM issue 1946).  max_pos must exceed every such position.
 * mt_rope_create allocates and synchronises the current device; destroy frees. */
typedef struct mt_rope mt_rope;
int mt_rope_create(double base, int head_dim, int max_pos, mt_rope** out);
int mt_rope_destroy(mt_rope* rope);

/* ---- Tree attention -------------------------------------------------------
 * For each sequence b, tree node i and query head h (KV head h / (Hq/Hkv)):
 *   out[b][i][h] = sum_j softmax_j(q'.k_j * sm_scale) v_j
 * over the keys j = prefix slots 0 .. L_b-1 of the paged cache, plus the tree
 * keys of i's ancestors, i itself included.  q' and the tree keys are rotated
 * at position L_b + depth[i]; the prefix keys are used as stored.  Before the
 * attention, node i's rotated key and raw value are written to logical slot
 * L_b + i (the scratch region), where mt_kv_commit later finds them; slots
 * below L_b are never written.  Accumulation in fp32, output rounded to nearest
 * even in the act dtype.  Where the schedule splits a (sequence, KV head) into
 * pieces, each piece's own softmax output is rounded to the act dtype first
 * and the fp32 merge is rounded again (the same tolerance holds).
 *   q      [B][T][Hq][D]    act   (not rotated)
 *   k_new  [B][T][Hkv][D]   act   (the tree tokens' keys, not rotated)
 *   v_new  [B][T][Hkv][D]   act
 *   k_cache, v_cache        act   paged layout above (written: scratch slots)
 *   block_tables, seq_lens  int32 (read only)
 *   tree_parents, tree_depths int32 [B][T]
 *   out    [B][T][Hq][D]    act
 *   workspace: device memory of mt_tree_attn_workspace_size(desc) bytes,
 *     zero-filled before its first use; it holds the device status word, the
 *     ancestor bitmasks, the schedule and the split-KV partial results.  One
 *     workspace per stream: calls sharing a workspace must not overlap. */
size_t mt_tree_attn_workspace_size(const mt_attn_desc* desc);
int mt_tree_attn_paged(const mt_attn_desc* desc, const void* q, const void* k_new,
                       const void* v_new, void* k_cache, void* v_cache,
                       const int32_t* block_tables, const int32_t* seq_lens,
                       const int32_t* tree_parents, const int32_t* tree_depths,
                       const mt_rope* rope, void* out, void* workspace, size_t ws_bytes,
                       cudaStream_t stream);

/* ---- Tree attention without allocation -------------------------------------
 * The pages this library follows have no counterpart for this call.  It is for
 * callers that cannot allocate device memory on the calling path -- for
 * example a serving loop that must not risk the device synchronisation and
 * out-of-memory failures of cudaMalloc between steps, or code that is handed
 * only its input and output buffers by a memory pool it does not own.
 * Same computation, arguments and layouts as mt_tree_attn_paged, but no
 * workspace argument: the workspace is a fixed 64 MiB array that the library
 * reserves on every device it is loaded on, held until the process exits.
 *  - Returns MT_ERR_UNSUPPORTED when mt_tree_attn_workspace_size(desc) exceeds
 *    64 MiB (e.g. very large batches; use mt_tree_attn_paged there).
 *  - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *  - The first call on a device, with that device current, looks up the
 *    array's device address (cudaGetSymbolAddress) and keeps it; make that
 *    first call before any stream capture.
 *  - All calls on one device share the array: calls that overlap on the GPU
 *    race, so issue them on one stream or order them with events.
 *  - Each call clears the array's device status word first; if device_status
 *    is not NULL (a device int32), the status after this call's kernels is
 *    copied there on `stream` (MT_OK or the device-detected error). */
int mt_tree_attn_paged_noalloc(const mt_attn_desc* desc, const void* q, const void* k_new,
                               const void* v_new, void* k_cache, void* v_cache,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               const int32_t* tree_parents, const int32_t* tree_depths,
                               const mt_rope* rope, void* out, int32_t* device_status,
                               cudaStream_t stream);

/* ---- Greedy acceptance ----------------------------------------------------
 * Per sequence b (LM head at temperature 0):
 *   argmax_out[b][i] = argmax_v target_logits[b][i][v], the lowest index among
 *                      equal maxima (values compared exactly; +0 equals -0);
 *   node 0 is accepted; node i > 0 is accepted when its parent is and
 *     tree_tokens[b][i] == argmax_out[b][parent[i]];
 *   end = the accepted node of largest depth, the lowest index among equals;
 *   accept_len[b]  = depth of end (accepted tokens besides the root);
 *   accept_path[b] = node ids root .. end, then -1, max_depth+1 entries;
 *   next_token[b]  = argmax_out[b][end], the token the target model adds.
 *   tree_tokens int32 [B][T]; target_logits [B][T][V] in logits_dtype (no NaN);
 *   tree_parents int32 [B][T]; every depth must be <= max_depth.
 *   workspace: mt_tree_accept_workspace_size(B, T) bytes, zero-filled before
 *   first use (status word, per-sequence arrival counters, which every call
 *   leaves at zero, per-node scratch for typical acceptance, and, for rows
 *   split over several CTAs when the rows are few, a per-row key and counter,
 *   also left at zero, and per-slice statistics). */
size_t mt_tree_accept_workspace_size(int batch, int tree_size);
int mt_tree_accept_greedy(int batch, int tree_size, int vocab, int max_depth,
                          mt_dtype logits_dtype, const int32_t* tree_tokens,
                          const void* target_logits, const int32_t* tree_parents,
                          int32_t* argmax_out, int32_t* accept_len, int32_t* accept_path,
                          int32_t* next_token, void* workspace, size_t ws_bytes,
                          cudaStream_t stream);

/* ---- Typical acceptance ---------------------------------------------------
 * The "typical acceptance scheme" that the opening comment of vLLM issue 1171
 * (gesanqiu: tree attention and typical acceptance are what most inference
 * frameworks lack) names beside tree attention; the pages do not define it, and
 * the rule taken is the Medusa paper's (Cai et al. 2024, typical acceptance).
 * Per sequence b, with x the logits row of a node and tau = temperature:
 *   q_v = exp(x_v / tau) / sum_u exp(x_u / tau), H = -sum_v q_v ln q_v;
 *   node i > 0 passes when q[tree_tokens[b][i]] > min(epsilon, delta * exp(-H))
 *     under its parent's row (a token outside [0, vocab) fails); the root
 *     passes; node_accept[b][i] = 1 when node i passes (its own test);
 *   accept_len, accept_path: as in mt_tree_accept_greedy with "accepted" =
 *     every node on the root path passes;
 *   next_token[b] = argmax of the end node's row (lowest index among equal
 *     maxima): the bonus token at temperature 0, no random draw.
 * Computed in fp32: the device sums the row in an order of its own, so a
 * node whose q[token] lies within a relative 1e-5 or so of its threshold may
 * fall either way.  temperature, epsilon, delta: positive and finite
 * (MT_ERR_INVALID_ARG otherwise; also when log2(e) / temperature overflows).
 * Logits: finite, and finite after scaling by log2(e) / temperature.
 * Layouts, max_depth and the workspace as for mt_tree_accept_greedy (the
 * same mt_tree_accept_workspace_size); node_accept int32 [B][T]. */
int mt_tree_accept_typical(int batch, int tree_size, int vocab, int max_depth,
                           mt_dtype logits_dtype, const int32_t* tree_tokens,
                           const void* target_logits, const int32_t* tree_parents,
                           float temperature, float epsilon, float delta, int32_t* node_accept,
                           int32_t* accept_len, int32_t* accept_path, int32_t* next_token,
                           void* workspace, size_t ws_bytes, cudaStream_t stream);

/* ---- KV commit --------------------------------------------------------------
 * For each sequence b, with L = accept_len[b] and len = seq_lens[b]:
 *   for d = 0..L: every KV head's K and V row at logical slot
 *     len + accept_path[b][d] is copied to slot len + d (all sources of a
 *     sequence are read before any destination is written);
 *   seq_lens[b] = len + L + 1;
 *   every logical block p with p*P >= len + L + 1 and p*P < len + T (tree
 *     scratch past the new length) is released: block_tables[b][p] becomes -1
 *     and its page id is listed, in ascending p, in released_pages[b][*], a row
 *     of (T + 2P - 2) / P entries padded with -1.
 *   accept_path int32 [B][max_depth+1], accept_len int32 [B] (as produced by
 *   mt_tree_accept_greedy); k_cache, v_cache, block_tables, seq_lens are
 *   updated in place.  desc supplies B, T, Hkv, D, P, max_blocks_per_seq,
 *   num_pages and the element size: dtype's, or 1 byte when cache_dtype is
 *   MT_E4M3 (the codes move unchanged).  status_ws: at least 256 bytes of device memory whose
 *   first int32 is the device status word (the attention workspace serves). */
int mt_kv_commit(const mt_attn_desc* desc, int max_depth, const int32_t* accept_path,
                 const int32_t* accept_len, void* k_cache, void* v_cache,
                 int32_t* block_tables, int32_t* seq_lens, int32_t* released_pages,
                 void* status_ws, cudaStream_t stream);

/* ---- Greedy acceptance and KV commit in one launch ---------------------------
 * The composition mt_tree_accept_greedy then mt_kv_commit (same results, same
 * arguments and layouts as those two calls), as one kernel launch: each
 * sequence is committed as soon as its path is known, by the CTA that
 * completed its argmax rows, so the step has no launch or round trip between
 * acceptance and commit.  desc supplies B (batch), T (tree_size), Hkv, D, P,
 * max_blocks_per_seq, num_pages and the cache's element size (as for
 * mt_kv_commit); the logits have their own dtype.  workspace: mt_tree_accept_workspace_size(B, T) bytes, zero-filled
 * before first use; its first int32 is the device status word, which records
 * the acceptance errors (MT_ERR_TREE) and the commit errors (MT_ERR_PAGES) of
 * both calls.  Host errors: those of the two calls.  A sequence whose tree is
 * malformed or too deep is accepted as the root alone (accept_len 0) and
 * committed so, exactly as the two calls would do. */
int mt_tree_accept_commit(const mt_attn_desc* desc, int vocab, int max_depth, mt_dtype logits_dtype,
                          const int32_t* tree_tokens, const void* target_logits,
                          const int32_t* tree_parents, int32_t* argmax_out, int32_t* accept_len,
                          int32_t* accept_path, int32_t* next_token, void* k_cache, void* v_cache,
                          int32_t* block_tables, int32_t* seq_lens, int32_t* released_pages,
                          void* workspace, size_t ws_bytes, cudaStream_t stream);

/* ---- Candidate tree tokens ---------------------------------------------------
 * The step before verification (lmdeploy PR 1231 "[WIP] support Medusa":
 * porting `generate_candidates`, Medusa heads at top-k over a 64-choice tree):
 * the tree's tokens from the base model's logits and the Medusa heads' logits.
 * For each sequence b, with the tree given by tree_parents[b] (node 0 the
 * root; parent[0] = -1, 0 <= parent[i] < i):
 *   tree_tokens[b][0] = argmax_v root_logits[b][v] (lowest index among equal
 *                       maxima);
 *   for node i >= 1 at depth d (1 <= d <= heads) with r earlier siblings (nodes
 *   j < i with the same parent): tree_tokens[b][i] = the entry of rank r
 *   (0-based) of head_logits[b][d-1], ordered by larger value first and lower
 *   vocab index first among equal values (+0 and -0 are equal); -1 when the
 *   head has fewer than r + 1 entries (r >= V).
 * root_logits [B][V] and head_logits [B][heads][V] in logits_dtype (no NaN);
 * tree_parents int32 [B][T]; tree_tokens int32 [B][T] out.  The tree template
 * (which choice of which head each node takes) is thus the tree's own shape:
 * the r-th child of a node takes the r-th best token of the next head.
 * Host errors: MT_ERR_INVALID_ARG for null or unaligned pointers or sizes out
 * of range (heads in [1, 63], V >= 1); MT_ERR_UNSUPPORTED for T outside
 * [1, 64] or another dtype.  Device status MT_ERR_TREE (in the first int32 of
 * status_ws, at least 256 bytes, read with mt_read_status): a malformed tree,
 * a node deeper than `heads`, or a node with 16 or more earlier siblings; the
 * tokens of that sequence (malformed tree or depth) or of that depth (too many
 * siblings) are not written.  The pages do not define the tree template; this
 * rule (child rank = head rank) is the reading used here. */
int mt_tree_candidates(int batch, int tree_size, int heads, int vocab, mt_dtype logits_dtype,
                       const void* root_logits, const void* head_logits,
                       const int32_t* tree_parents, int32_t* tree_tokens, void* status_ws,
                       cudaStream_t stream);

/* ---- Norms of queries and keys with the rotation ------------------------------
 * Not on the pages; for models whose attention normalises every query and key
 * head, and for the calls below, which take rotated rows.  For each token i and
 * each head row x of q and k, in fp32 with one rounding to the act dtype:
 *   y = x * rsqrt(mean(x^2) + eps) * weight   (weight act [D]; skipped when both
 *                                              weights are null)
 *   y rotated at positions[i] as defined above (skipped when rope is null).
 * positions int32 [num_tokens] (may be null without rope): a negative entry
 * marks a place without a token, whose rows of the outputs are left as they
 * were; one at or past the table's end is recorded as MT_ERR_POSITION in
 * status_ws (at least 256 bytes) and its rows are left as they were.
 * Strides are in elements, (token, head); each a whole number of 16 bytes, the
 * D elements of a row dense.  An output may be its own input (the same pointer
 * and strides); other overlaps are not supported. */
typedef struct {
  int num_tokens;
  int num_q_heads;
  int num_kv_heads;
  int head_dim;            /* 64 or 128 */
  mt_dtype dtype;
  float eps;
  long long q_stride[2];
  long long k_stride[2];
  long long q_out_stride[2];
  long long k_out_stride[2];
} mt_norm_rope_desc;
int mt_qk_norm_rope(const mt_norm_rope_desc* desc, const void* q, const void* k, const int32_t* positions,
                    const void* q_weight, const void* k_weight, const mt_rope* rope, void* q_out,
                    void* k_out, void* status_ws, cudaStream_t stream);

/* ---- Appending keys and values to the paged cache ------------------------------
 * How a prompt's rows, or an accepted path's, get into the pages.  New row i of
 * sequence b goes to logical slot seq_lens[b] + i; its key is rotated at that
 * position when rope is given (rounded once to the act dtype, the same
 * arithmetic as mt_tree_attn_paged), its value is stored as given.  seq_lens
 * and block_tables are read only: a model's layers append with the same lengths,
 * and the caller grows them once.
 *   mt_kv_append_paged     sequence b's new rows are k/v rows row_offsets[b] ..
 *                          row_offsets[b + 1] - 1 (int32 [B + 1], never falling,
 *                          within [0, num_rows]; other rows are ignored);
 *   mt_kv_append_accepted  k and v are the tree's rows [B][T] (num_rows = B * T)
 *                          and row i is node accept_path[b][i], i = 0 ..
 *                          accept_len[b] (as mt_tree_accept_greedy gives them):
 *                          the commit of a cache that mt_tree_attn_paged_block8
 *                          reads.
 * The cache holds the act dtype (cache_dtype 0), E4M3 codes of value / k_scale
 * and value / v_scale (MT_E4M3 without scale arrays), or E4M3 codes with a scale
 * for each block, one page of one KV head (MT_E4M3 with k_scales and v_scales,
 * fp32 [num_pages][Hkv]):
 *   scale = the smallest power of two 2^k, -64 <= k <= 119, with
 *           largest |value| of the block <= 448 * 2^k;
 *   a page that already holds older rows of its sequence keeps the larger of
 *   its scale and the new rows'; when that grows, the older rows' codes become
 *   the codes of (their value / the new scale), rounded to nearest even.
 * A NaN is stored as the NaN code and does not enter the scale; an infinity
 * makes the scale 2^119 and saturates.
 * A sequence with seq_lens[b] < 0 is no sequence: nothing is written for it.
 * Device status (status_ws, at least 256 bytes): MT_ERR_PAGES for offsets out of
 * range or falling, an accepted length or node out of range, a table that does not
 * cover the slots (nothing of that sequence is written; after falling offsets, of
 * later sequences perhaps not all), a page id out of range (nothing of that page is
 * written); MT_ERR_POSITION for a slot past the RoPE table (nothing of that
 * page is written).  A call must not append to a page twice: not for two
 * sequences, and not through a table that names the page twice.
 * Strides of k and v in elements, (row, head), whole numbers of 16 bytes. */
typedef struct {
  int batch;
  int num_rows;
  int num_kv_heads;
  int head_dim;            /* 64 or 128 */
  int page_size;           /* 16 */
  int max_blocks_per_seq;
  int num_pages;
  mt_dtype dtype;
  int cache_dtype;         /* 0 or MT_E4M3 */
  float k_scale;           /* MT_E4M3 without scale arrays */
  float v_scale;
  long long k_stride[2];
  long long v_stride[2];
} mt_append_desc;
int mt_kv_append_paged(const mt_append_desc* desc, const void* k, const void* v,
                       const int32_t* row_offsets, const mt_rope* rope, void* k_cache, void* v_cache,
                       float* k_scales, float* v_scales, const int32_t* block_tables,
                       const int32_t* seq_lens, void* status_ws, cudaStream_t stream);
int mt_kv_append_accepted(const mt_append_desc* desc, int tree_size, int max_depth, const void* k,
                          const void* v, const int32_t* accept_path, const int32_t* accept_len,
                          const mt_rope* rope, void* k_cache, void* v_cache, float* k_scales,
                          float* v_scales, const int32_t* block_tables, const int32_t* seq_lens,
                          void* status_ws, cudaStream_t stream);

/* ---- Tree attention over a block-scaled 8-bit cache ----------------------------
 * As mt_tree_attn_paged, with three differences:
 *   - the cache holds E4M3 codes with a scale for each (page, KV head), as
 *     mt_kv_append_paged writes them, and is only read: no scratch slots, and the
 *     table need cover slots 0 .. seq_lens[b] - 1 only;
 *   - q and k_new are rows as they attend (rotated by mt_qk_norm_rope);
 *   - the tree's own keys and values are seen as the append would encode them in
 *     blocks of 16 nodes (nodes 16j .. 16j + 15 of one KV head), as E4M3 codes with
 *     the block scale above.  (An accepted node's page has other rows and so perhaps
 *     another scale: its stored values differ where a code underflows under one of
 *     the two, here by way of large siblings that were rejected.)
 * T = 1 is a decoding step (tree_parents null, or -1); tree_parents null is a
 * chain, each node the child of the one before it.
 *   q [B][T][Hq][D], k_new, v_new [B][T][Hkv][D], out [B][T][Hq][D]  act (fp16 or bf16)
 *   k_cache, v_cache [num_pages][Hkv][16][D] codes; k_scales, v_scales fp32
 *   [num_pages][Hkv], of the range that the appends write, 2^-64 to 2^119 (powers
 *   of two or not); a value scale below it counts as 2^-64
 * A sequence with seq_lens[b] < 0 is no sequence: its rows of out are left as
 * they were.  desc: dtype MT_F16 or MT_BF16, cache_dtype MT_E4M3; num_splits,
 * kernel, k_scale and v_scale are not used; any number of query heads per KV
 * head.  out must not overlap q, k_new or v_new.  Accumulation in fp32.  A query's
 * elements keep their bits down to 2^-17 of the row's largest.  A key's softmax
 * weight times its block's value scale is rounded to fp16, relative to the largest
 * such product that the row sees: to 2^-11 of itself or, where it is small, to 2^-28
 * of the largest.  (Value scales some 2^100 apart in one sequence can cost the
 * smaller ones' keys their share of the sum of weights, too.)
 * A query row with a NaN or an infinity gives NaN, and so does a row that sees a
 * cached key with a NaN, or a new token with a NaN or an infinity in its key or
 * value; a cached value's NaN reaches its own column.  (A cached infinity is the
 * saturated code under the scale 2^119.)  NaN and infinities that a row does not see
 * have no effect on it: those of new tokens do not enter a block's scale.  A large
 * finite value that it does not see has one: it raises the scale of its block of 16
 * new tokens, so that the others' codes there are coarser.
 * workspace: mt_tree_attn_block8_workspace_size(desc) bytes, zero-filled before
 * its first use (status word, counters that every call leaves at zero, schedule,
 * partial results); it serves any descriptor that it is large enough for, one call
 * at a time: calls that share one, replays of captured ones too, must not overlap.
 * Device status: MT_ERR_PAGES (length past the table, page id
 * out of range), MT_ERR_TREE (a parent that is not earlier); the outputs of an
 * affected sequence are unspecified. */
size_t mt_tree_attn_block8_workspace_size(const mt_attn_desc* desc);
int mt_tree_attn_paged_block8(const mt_attn_desc* desc, const void* q, const void* k_new,
                              const void* v_new, const void* k_cache, const void* v_cache,
                              const float* k_scales, const float* v_scales,
                              const int32_t* block_tables, const int32_t* seq_lens,
                              const int32_t* tree_parents, void* out, void* workspace,
                              size_t ws_bytes, cudaStream_t stream);

/* ---- Sampling --------------------------------------------------------------------
 * A drawn token beside the argmax that greedy and typical acceptance return (the
 * bonus token of an accepted path's last row, or a decoding step's).  For each i,
 * with x the logits row row_index[i] (row i when row_index is null), m its
 * maximum and t = temperature[i]:
 *   w_v = exp((x_v - m) / t); the tokens are ordered by larger x, then lower
 *   index; kept are those among the first top_k[i], with (mass before them) <
 *   top_p[i] * (mass of the first top_k[i]), and with w_v >= min_p[i]; the first
 *   is always kept; tokens[i] = the lowest v for which the kept mass of tokens
 *   0 .. v exceeds uniforms[i] * (kept mass).
 * t <= 0: the argmax (lowest index among equals).  top_k <= 0 or >= vocab,
 * top_p >= 1, min_p <= 0: off.  A null parameter array: temperature 1, filters
 * off.  uniforms: numbers of [0, 1), others are clamped.  A NaN logit counts as
 * -inf; a row without anything above -inf gives -1; entries of +inf share the
 * whole mass.  Weights are cut to whole multiples of 2^-44 of the largest and are
 * good to 1e-9 of themselves besides; their sums are exact (2^-38 for the cut by
 * top_p).  So the token is that of the definition unless u or top_p times its mass
 * lies next to a border: by 1e-9 of the mass and vocab * 2^-44 of the largest weight
 * (3e-8 for 500000 tokens).
 * row_index[i] < 0: no row, tokens[i] is left as it was; >= num_logit_rows: -1.
 * row_stride in elements; rows need no alignment.  vocab <= 500000
 * (MT_ERR_UNSUPPORTED above).  No workspace and no device status. */
int mt_sample_tokens(int num_rows, int vocab, mt_dtype logits_dtype, const void* logits,
                     int num_logit_rows, long long row_stride, const int32_t* row_index,
                     const float* uniforms, const float* temperature, const int32_t* top_k,
                     const float* top_p, const float* min_p, int32_t* tokens, cudaStream_t stream);

/* ---- Status ------------------------------------------------------------------
 * Waits for `stream`, then reads and clears the device status word at the start
 * of `workspace` (MT_OK or the first device-side error since the last read). */
int mt_read_status(void* workspace, cudaStream_t stream, int* device_status);
const char* mt_status_string(int status);

/* ---- Profiling hook -----------------------------------------------------------
 * mt_profile_enable(n) creates n pairs of CUDA events (0 disables and frees
 * them).  While fewer than n pairs are used, each mt_tree_attn_paged call
 * records one pair on its stream, immediately around its main attention kernel
 * (the ancestor/scatter preparation and the split-KV combine are outside it).
 * mt_profile_read waits for the recorded pairs, writes their elapsed times in
 * milliseconds to ms[0 .. *n_out-1] and starts over.  Not thread-safe: for one
 * host thread driving the library. */
int mt_profile_enable(int max_records);
int mt_profile_read(float* ms, int max_records, int* n_out);

/* ---- Timeout test hook --------------------------------------------------------
 * Every pipeline wait of the tensor-core attention kernels (a TMA load landing,
 * an MMA completing, a softmax handing over P) gives up after a bounded time:
 * the kernel then records MT_ERR_TIMEOUT in the status word, lets its other
 * warps stop, waits for its own copies and MMAs in flight, frees its tensor
 * memory and returns, leaving the context usable.  mt_debug_set_wait sets that
 * bound for later mt_tree_attn_paged and mt_tree_attn_paged_block8 calls (limit_ns 0 restores the default of
 * 2 s); stall = 1 makes the kernel first wait on a barrier that nothing
 * completes, so that the bound always expires (for tests of the timeout path;
 * stall = 0 is normal operation).  Process-wide, not thread-safe.  Returns
 * MT_ERR_INVALID_ARG for a stall other than 0 or 1.  Not on the pages: the
 * wait bound is how this library reports a stalled pipeline instead of
 * hanging the GPU. */
int mt_debug_set_wait(unsigned long long limit_ns, int stall);

/* Version of this ABI: major * 10000 + minor * 100 + patch. */
int mt_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MEDUSA_TREE_H_ */
