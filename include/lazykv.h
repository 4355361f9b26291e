/*
 * lazykv.h -- C ABI of liblazykv.so: LazyAttention's hot path on one GB300 (sm_103a).
 *
 * LazyAttention ("LazyAttention: Efficient Retrieval-Augmented Generation with Deferred
 * Positional Encoding", ICML 2026) keeps ONE position-free KV copy per document and applies
 * the positional encoding inside the attention kernels.  Sources cited below:
 *   [NOTE]   papernotes.org reading note on the paper: sections 方法详解/整体框架
 *            (position-free cache, Example 3.1), 关键设计 (Deferred Positional Encoding;
 *            Tiling 感知的 Q/K 旋转分派; 融合 Triton kernel + bit-packed 元数据), 通用性.
 *   [GIST]   gist.science technical summary: Implementazione Tecnica (Prefilling,
 *            Decoding), Equivalenza Matematica.
 *   [README] illinoisdata/lazy-attention README mirror: Variants (scheduler metadata).
 *
 * Conventions for every entry point
 *   - Pointers marked (host) are CPU memory; (device) are GPU memory the CALLER allocated
 *     (e.g. by PyTorch) and owns.  The library allocates no device memory and keeps no state
 *     beyond one 32-bit device status word per GPU (see lazy_device_status).
 *   - bf16 tensors are contiguous, row-major, 16-byte aligned.
 *   - Paged caches: k_cache and v_cache are bf16 [num_pages][Hkv][16][D]; one page of one KV
 *     head is 16 * D * 2 bytes, contiguous.  A cache slot is page * 16 + row.  The attention
 *     kernels read only rows that hold a key the query can see (a block's first n_valid rows,
 *     and in the query segment none past the query's position), so the rest of a page may hold
 *     anything, uninitialised or NaN bits included.
 *   - Every GPU entry point is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream), performs no synchronisation and returns after the launch.
 *   - Kernels are launched with programmatic dependent launch: one may become resident while
 *     the previous kernel of the stream drains, and it reads or writes no global memory until
 *     that kernel has completed (griddepcontrol.wait), so stream order is kept exactly as for
 *     a plain launch, including inside CUDA graph capture.
 *   - Return codes: LAZY_OK, or a negative code with a message for lazy_last_error().
 *     Argument errors are detected on the host before anything is launched.  Errors found
 *     by a kernel (an out-of-range page or slot, a wait that ran out) set bits of the device
 *     status word and the offending element is skipped; no kernel traps or asserts.
 *   - Head dims supported: D in {64, 128}; rotary_dim a multiple of 16 in [16, D] (RoPE and
 *     YaRN).  Hq % Hkv == 0.
 */
#ifndef LAZYKV_H
#define LAZYKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LAZY_OK 0
#define LAZY_EINVAL (-1) /* shape, pointer, alignment or dtype argument not supported     */
#define LAZY_ERANGE (-2) /* a value does not fit a field of the 64-bit block word, or max_blocks too small */
#define LAZY_ECUDA (-3)  /* a CUDA runtime call or kernel launch failed                   */
#define LAZY_EARCH (-4)  /* the current GPU is not compute capability 10.x                */
#define LAZY_EDEVICE (-5) /* a kernel reported an error through the device status word    */

#define LAZY_PAGE_SIZE 16

/* Device status word bits (lazy_device_status). */
#define LAZY_STATUS_BAD_PAGE 1u    /* a block word named a page >= num_pages            */
#define LAZY_STATUS_BAD_SLOT 2u    /* kv_write got a slot outside the caches             */
#define LAZY_STATUS_TIMEOUT 4u     /* a bounded wait on a copy or MMA ran out            */
#define LAZY_STATUS_BAD_ROW 8u     /* a query row's visible range exceeded max_blocks    */

/* Positional encodings ([NOTE] 通用性: RoPE variants and ALiBi change only metadata). */
enum {
  LAZY_POS_ROPE = 0,  /* RoPE, theta_i = rope_theta^(-2i/rotary_dim); half-split pairs
                         (x_i, x_{i+rotary_dim/2}) or interleaved (x_2i, x_2i+1)          */
  LAZY_POS_YARN = 1,  /* YaRN-scaled RoPE frequencies (YaRN paper's ramp) + mscale^2     */
  LAZY_POS_ALIBI = 2, /* no rotation; logit += -alibi_slopes[h] * (m - p)                */
  LAZY_POS_NONE = 3   /* no positional work at all: the "Delta = 0" twin used to time the
                         cost of deferred rotation (same kernels, rotation compiled out)  */
};

/*
 * Positional configuration, read on the host at call time (by value semantics).
 *   rope_theta, rotary_dim          RoPE base and rotated width: the first rotary_dim
 *                                   dimensions of every head are rotated, the rest pass
 *                                   through (a multiple of 16 in [16, D]).
 *   yarn_factor, yarn_orig_ctx,     YaRN scale s, original context L0, ramp bounds
 *   yarn_beta_fast, yarn_beta_slow  (defaults 32 and 1 when given as 0).
 *   alibi_slopes                    (device) float [Hq]; ALiBi only.
 *   cos_sin                         (device) float [max_pos][rotary_dim] table written by
 *                                   lazy_build_rope_table (cos in the first half of a row,
 *                                   sin in the second), or NULL: compute cos/sin on the fly.
 *   max_pos                         rows of cos_sin.
 *   interleaved                     0: half-split pairs (x_i, x_{i + rotary_dim/2}) (NeoX /
 *                                   Llama); 1: adjacent pairs (x_2i, x_2i+1) (GPT-J).  The
 *                                   pages treat RoPE variants as metadata ([NOTE] 通用性).
 */
typedef struct lazy_pos_cfg {
  int32_t kind;
  int32_t rotary_dim;
  float rope_theta;
  float yarn_factor;
  int32_t yarn_orig_ctx;
  float yarn_beta_fast;
  float yarn_beta_slow;
  const float* alibi_slopes;
  const float* cos_sin;
  int32_t max_pos;
  int32_t interleaved;
} lazy_pos_cfg;

/*
 * lazy_build_doc_meta -- per-request block list with one packed 64-bit word per block.
 * [README] Variants (the scheduler builds rotation metadata); [NOTE] 融合 Triton kernel +
 * bit-packed 元数据 (block id, offset and mask in one 64-bit register); [NOTE] 整体框架
 * (each document indexed from local position 0; the request places it at offset Delta).
 *
 * All pointers (host).  Request b lists documents req_docs[req_doc_off[b] .. req_doc_off[b+1]),
 * each an index into doc_len [n_docs] and the page lists doc_pages[doc_page_off[d] ..
 * doc_page_off[d+1]).  Its query segment (prefill tokens then decode tokens) has q_len[b]
 * prefill tokens and capacity pages q_pages[q_page_off[b] .. q_page_off[b+1]).
 * Outputs, each [B][max_blocks] or [B], fully written (unused tail entries = 0):
 *   block_table  int32  physical page of each block
 *   meta         uint64 word: bits [4:0] n_valid (1..16), [15:5] page index within the
 *                document pg (< 2048), [39:16] Delta (< 2^24), [63:40] physical page (< 2^24).
 *                Key row t of a block sits at absolute position p = Delta + 16 * pg + t.
 *                Query-segment blocks are listed as full (n_valid = 16); causality (p <= m)
 *                masks their unwritten rows, and the attention kernels never read them.
 *   seq_len      keys visible after the prefill tokens are written (= q_start + q_len)
 *   q_start      Delta of the query segment (= total document length)
 *   doc_blocks   number of document blocks (the query segment starts at this block)
 * Returns LAZY_EINVAL for negative lengths or missing pages, LAZY_ERANGE when a field
 * overflows or a request needs more than max_blocks blocks.  Deterministic, bit-exact.
 */
int lazy_build_doc_meta(int B, const int32_t* req_doc_off, const int32_t* req_docs, int n_docs,
                        const int32_t* doc_len, const int32_t* doc_page_off,
                        const int32_t* doc_pages, const int32_t* q_len,
                        const int32_t* q_page_off, const int32_t* q_pages, int max_blocks,
                        int32_t* block_table, uint64_t* meta, int32_t* seq_len,
                        int32_t* q_start, int32_t* doc_blocks);

/*
 * lazy_build_rope_table -- cos/sin table for the positional config ([NOTE] Tiling 感知:
 * cos/sin read from a table, one D-length vector per document offset).
 * out_table (device) float [max_pos][rotary_dim]: row p holds cos(p theta_i) for i < d/2,
 * then sin(p theta_i).  Angles are reduced exactly (fixed-point turn count), so row p is
 * accurate to ~2e-7 for every p < 2^24.  ALiBi / NONE: LAZY_EINVAL.
 */
int lazy_build_rope_table(const lazy_pos_cfg* cfg, int max_pos, float* out_table, void* stream);

/*
 * lazy_kv_write -- write T tokens into the paged caches, position-free ([NOTE] 整体框架:
 * the cache holds content indexed from each document's local position 0).
 *   k, v       (device) bf16 [T][Hkv][D], raw (pre-RoPE) keys and values
 *   slot       (device) int32 [T], page * 16 + row of each token
 *   local_pos  (device) int32 [T], position j of the token inside its document / segment
 * Stored K = bf16_RNE(R_j k) computed in fp32 (RoPE/YaRN); raw k for ALiBi/NONE.
 * Stored V = v.  A slot outside [0, num_pages * 16) sets LAZY_STATUS_BAD_SLOT and the token
 * is skipped.
 */
int lazy_kv_write(const void* k, const void* v, const int32_t* slot, const int32_t* local_pos,
                  int T, int Hkv, int D, void* k_cache, void* v_cache, int num_pages,
                  const lazy_pos_cfg* cfg, void* stream);

/*
 * lazy_attn_decode -- one decode step (M = 1 per request), GQA-grouped, split over the KV
 * sequence.  [NOTE] Tiling 感知的 Q/K 旋转分派: decode rotates Q, and only when the KV block
 * crosses a document boundary; [NOTE] 融合 Triton kernel: the block word is unpacked from a
 * register; [GIST] Decoding.
 *   q          (device) bf16 [B][Hq][D] raw queries; request b's query sits at
 *              m = seq_len[b] - 1 and its own key/value were written at p = m beforehand
 *   seq_len, q_start, doc_blocks  (device) int32 [B] from lazy_build_doc_meta (seq_len
 *              advanced by the caller for every decode token written)
 *   meta       (device) uint64 [B][max_blocks]
 *   scale      softmax scale; 0 selects 1/sqrt(D) (times mscale^2 for YaRN)
 *   out        (device) bf16 [B][Hq][D];  lse (device, nullable) float [B][Hq], natural log
 *   ws         (device) workspace of at least lazy_workspace_size(LAZY_PHASE_DECODE, ...)
 *              bytes, 256-byte aligned, or NULL when that size is 0.
 * Keys visible to m: every document block plus the query segment up to p <= m.
 */
int lazy_attn_decode(const void* q, const int32_t* seq_len, const int32_t* q_start,
                     const int32_t* doc_blocks, const uint64_t* meta, int B, int max_blocks,
                     const void* k_cache, const void* v_cache, int num_pages, int Hq, int Hkv,
                     int D, float scale, const lazy_pos_cfg* cfg, void* out, float* lse,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * lazy_attn_decode_noalloc -- lazy_attn_decode for callers that cannot allocate device memory.
 * The paper has no counterpart: this is a deployment variant of the decode above.
 *
 * Who needs it: a host that owns all GPU memory itself (e.g. an engine that reserves HBM for
 * its KV pool at start-up and gives plugins no allocator), or a latency-bound loop that must
 * never call cudaMalloc (which can synchronise the device).  Such callers cannot pass the
 * split-KV workspace lazy_attn_decode needs, so this entry point uses a fixed 16 MiB array
 * compiled into the library instead; neither the caller nor the library allocates (no
 * cudaMalloc, cudaFree or allocating library routine is called).
 *   Arguments, layouts and results: exactly those of lazy_attn_decode, without ws/ws_bytes.
 *   Limit: batches whose split scratch (see lazy_workspace_size) exceeds 16 MiB are rejected
 *          with LAZY_EINVAL and a message; nothing is launched.
 *   Memory: every GPU that loads the library holds the 16 MiB array until the process exits.
 *   Set-up: the first call on each device looks up the array's device address (with that
 *          device current); make that first call before any stream capture.
 *   Sharing: all calls on a device share the one array and it keeps the last call's contents.
 *          Nothing in it must start at zero.  Calls that overlap on the GPU (different
 *          streams, or different host threads) race on it: serialise them.
 */
int lazy_attn_decode_noalloc(const void* q, const int32_t* seq_len, const int32_t* q_start,
                             const int32_t* doc_blocks, const uint64_t* meta, int B,
                             int max_blocks, const void* k_cache, const void* v_cache,
                             int num_pages, int Hq, int Hkv, int D, float scale,
                             const lazy_pos_cfg* cfg, void* out, float* lse, void* stream);

/*
 * lazy_attn_prefill -- causal prefill of every request's query tokens over its documents and
 * its own earlier tokens.  [NOTE] Tiling 感知: prefill rotates each K tile by its document's
 * Delta (Q tiles are much taller than K tiles); [NOTE] 融合 Triton kernel (K tile split in
 * halves, rotated per half-dimension, then the GEMM); [GIST] Prefilling.
 *   q          (device) bf16 [total_q][Hq][D] raw queries; rows cu_q[b] .. cu_q[b+1] belong
 *              to request b and sit at absolute positions q_start[b] + i.  Their keys and
 *              values must already be in the cache (lazy_kv_write with local_pos = i).
 *   cu_q       (device) int32 [B+1];  max_q = max_b (cu_q[b+1] - cu_q[b]) (host value)
 *   out        (device) bf16 [total_q][Hq][D];  lse (device, nullable) float [total_q][Hq]
 *   ws / ws_bytes as for decode, sized by lazy_workspace_size(LAZY_PHASE_PREFILL, ...).
 */
int lazy_attn_prefill(const void* q, const int32_t* cu_q, const int32_t* q_start,
                      const int32_t* doc_blocks, const uint64_t* meta, int B, int max_blocks,
                      int total_q, int max_q, const void* k_cache, const void* v_cache,
                      int num_pages, int Hq, int Hkv, int D, float scale,
                      const lazy_pos_cfg* cfg, void* out, float* lse, void* ws,
                      size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * 4-bit caches.  The same paged, position-free cache (one copy of a document, keys rotated by
 * their local positions) in 4.5 bits per value instead of 16: every 16 consecutive dimensions
 * of a row form a group with one e4m3 scale s, and a value is an e2m1 code (sign, then 0, 0.5,
 * 1, 1.5, 2, 3, 4 or 6) times s times the cache's factor (k_scale / v_scale, a power of two in
 * [2^-32, 2^32]; 0 selects 1).  s = e4m3(max |y| / (6 factor)), at most 448; the code is the
 * nearest of y / factor / s, ties to even, saturating at 6.  A group with an infinity or a NaN
 * gets the scale NaN and reads back as NaN.  Choose a factor other than 1 only if a group's
 * maximum can leave [0.1, 2688]: smaller ones lose accuracy in s, larger ones saturate.  All
 * calls on a cache take the same factors.
 *
 * kv_cache (device) uint8 [num_pages][Hkv][18 D], 16-byte aligned: one block of 18 D bytes per
 * page and KV head.  For row r (0..15) and dimension d of a block:
 *   K code   r D/2 + d/2 (low half of the byte: even d)
 *   K scale  8 D + ((r % 8) 4 + d / (D/4)) D/32 + (r / 8) D/64 + (d % (D/4)) / 16
 *   V code   9 D + (r / 8) A + (d / (D/8) 4 + (r % 8) / 2) 16 + (r % 2) D/16 + (d % (D/8)) / 2,
 *            A = 512 for D = 128 and 8 for D = 64 (low half of the byte: even d)
 *   V scale  17 D + (d / 16) 16 + ((r % 8) / 2) 4 + (r / 8) 2 + r % 2
 * Rows that hold no visible key may hold anything; a NaN makes NaN only of the query rows that see
 * it (in a key: all of their outputs for its KV head, in a value: those of its group).  Slots, block
 * words, query and workspace conventions are those of the bf16 entry points above; so are the head
 * shapes they accept, the status bits and the return codes.  Arguments are checked before the
 * device is.
 * ------------------------------------------------------------------------------------------ */

/*
 * lazy_kv_write_q4 -- lazy_kv_write into a 4-bit cache: quantises bf16_RNE(R_j k) and v.  With a
 * cos/sin table in cfg the rotation is fl(fl(x1 c) - fl(x2 s)), fl(fl(x1 s) + fl(x2 c)) in fp32.
 * Only the bytes of the written rows change.  The slots of one call must be distinct: a row
 * that two tokens share ends as a mix of both.
 */
int lazy_kv_write_q4(const void* k, const void* v, const int32_t* slot, const int32_t* local_pos,
                     int T, int Hkv, int D, void* kv_cache, int num_pages,
                     const lazy_pos_cfg* cfg, float k_scale, float v_scale, void* stream);

/*
 * lazy_kv_read_q4 -- the values held in T cache rows, exactly, in bf16 (keys as stored: rotated
 * by their local positions).
 *   slot  (device) int32 [T];  k, v  (device, written) bf16 [T][Hkv][D]
 * A slot outside [0, num_pages * 16) sets LAZY_STATUS_BAD_SLOT and its output rows are left as
 * they were.
 */
int lazy_kv_read_q4(const int32_t* slot, int T, int Hkv, int D, const void* kv_cache,
                    int num_pages, float k_scale, float v_scale, void* k, void* v, void* stream);

/*
 * lazy_attn_decode_q4 / lazy_attn_prefill_q4 -- lazy_attn_decode / lazy_attn_prefill over a
 * 4-bit cache.  Workspace: lazy_workspace_size with LAZY_PHASE_DECODE_Q4 / LAZY_PHASE_PREFILL_Q4.
 * A row without a visible key gets out = 0 and lse = -inf; rows of q outside [cu_q[0], cu_q[B])
 * (a batch padded to a fixed size) keep what out and lse held.  max_q may be any upper bound of the
 * requests' query rows.  A negative or non-finite scale is
 * refused, and one whose product with k_scale (0: the default 1/sqrt(D); with YaRN's factor and
 * log2 e) lies outside [2^-60, 2^60].
 */
int lazy_attn_decode_q4(const void* q, const int32_t* seq_len, const int32_t* q_start,
                        const int32_t* doc_blocks, const uint64_t* meta, int B, int max_blocks,
                        const void* kv_cache, int num_pages, int Hq, int Hkv, int D, float scale,
                        float k_scale, float v_scale, const lazy_pos_cfg* cfg, void* out,
                        float* lse, void* ws, size_t ws_bytes, void* stream);
int lazy_attn_prefill_q4(const void* q, const int32_t* cu_q, const int32_t* q_start,
                         const int32_t* doc_blocks, const uint64_t* meta, int B, int max_blocks,
                         int total_q, int max_q, const void* kv_cache, int num_pages, int Hq,
                         int Hkv, int D, float scale, float k_scale, float v_scale,
                         const lazy_pos_cfg* cfg, void* out, float* lse, void* ws,
                         size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Batches that share documents, and eviction inside a context (bf16 caches).  Slots, block words,
 * query and workspace conventions are those of the entry points above; so are the status bits and the
 * return codes.  Arguments are checked before the device is.  cfg->cos_sin is not read: angles come from
 * exact turn counts.  A negative or non-finite scale is refused, and one that (0: the default 1/sqrt(D),
 * with YaRN's factor; times log2 e) lies outside [2^-60, 2^60].  Hq / Hkv may be any whole number.
 * ------------------------------------------------------------------------------------------ */

/*
 * lazy_attn_decode_shared -- lazy_attn_decode for a batch in which groups of requests list the same first
 * documents: their common keys are read once per group instead of once per request.
 *   group_off      (device) int32 [n_groups + 1], not decreasing: requests group_off[g] ..
 *                  group_off[g+1]-1 form group g; requests outside every group are decoded alone
 *   shared_blocks  (device) int32 [n_groups]: the first shared_blocks[g] words of the group's lists are the
 *                  same; document blocks only (at most the doc_blocks of each of its requests).  They are
 *                  read from the list of the group's first request (which holds them even if it is idle).
 *   max_group      upper bound (host) of the groups' sizes
 *   max_shared     upper bound (host) of shared_blocks; a larger group or value is cut to it (with
 *                  LAZY_STATUS_BAD_ROW), and what is cut off is decoded alone: the results are the same
 *   ws             lazy_decode_shared_workspace_size bytes, 256-byte aligned
 * q, seq_len, q_start, doc_blocks, meta, out and lse as in lazy_attn_decode.  seq_len[b] <= 0 marks an idle
 * request (a batch padded to a fixed size); it and one without a visible key get out = 0 and lse = -inf.
 * Common keys are rotated and taken in f16 (as in lazy_attn_prefill: magnitudes above 65504 overflow); a NaN
 * or an infinity in a common value reaches that column of every request of the group.  Few and short lists are decoded one by
 * one, where that is faster; a long list of a request alone is best given as a group of one.
 */
int lazy_attn_decode_shared(const void* q, const int32_t* seq_len, const int32_t* q_start,
                            const int32_t* doc_blocks, const uint64_t* meta, const int32_t* group_off,
                            const int32_t* shared_blocks, int n_groups, int max_group, int max_shared, int B,
                            int max_blocks, const void* k_cache, const void* v_cache, int num_pages, int Hq,
                            int Hkv, int D, float scale, const lazy_pos_cfg* cfg, void* out, float* lse,
                            void* ws, size_t ws_bytes, void* stream);

/* Bytes of workspace of a lazy_attn_decode_shared call with these sizes (query it with the device that
 * will run the call current). */
size_t lazy_decode_shared_workspace_size(int B, int n_groups, int max_group, int max_shared, int max_blocks,
                                         int Hq, int Hkv, int D);

/*
 * lazy_attn_key_weights -- the attention weight that every cached key receives:
 *   weights[b][16 j + t] (+)= sum over query rows i and heads h of exp(scale q_ih . R k - lse_ih)
 * for the key in row t of the request's j-th block, over the rows that see it.
 *   q        (device) bf16 [total_q][Hq][D] raw queries; rows cu_q[b] .. cu_q[b+1] are the last tokens of
 *            request b, the last of them at position seq_len[b] - 1 (a decode step: cu_q[b] = b; a prefill:
 *            its own cu_q, and seq_len from lazy_build_doc_meta)
 *   lse      (device) float [total_q][Hq], from the attention call over the same list
 *   max_q    upper bound (host) of the rows of a request; of more rows the last max_q count
 *            (LAZY_STATUS_BAD_ROW)
 *   window   > 0: only the last `window` rows of each request count; 0: all of them
 *   accumulate  0: weights is written, 0 where no key lies; 1: added to
 *   weights  (device) float [B][16 max_blocks]
 *   ws       lazy_workspace_size(LAZY_PHASE_KEY_WEIGHTS, ...) bytes, 256-byte aligned
 * A row with lse = -inf (nothing visible) counts nothing, a NaN key takes its own weight, a NaN row those of
 * the keys that it sees.  Queries count with 24 bits where max_q and window leave a request up to 32 rows per KV
 * head, else with 16: a tight max_q is worth giving.  Sums are in fp32 and in a fixed order: two calls give the
 * same bits.
 */
int lazy_attn_key_weights(const void* q, const float* lse, const int32_t* cu_q, const int32_t* seq_len,
                          const int32_t* q_start, const int32_t* doc_blocks, const uint64_t* meta, int B,
                          int max_blocks, int total_q, int max_q, int window, const void* k_cache,
                          int num_pages, int Hq, int Hkv, int D, float scale, const lazy_pos_cfg* cfg,
                          int accumulate, float* weights, void* ws, size_t ws_bytes, void* stream);

/*
 * lazy_evict_plan -- which document keys of each request stay, and where they go.  A stored key carries its
 * rotation by its position in the document and attention adds the document's, so a key may move to any row
 * of a page with the same Delta: keys that stay are packed document by document into new pages, in order,
 * and keep their positions.  (With ALiBi the position is the row's: refused.)
 *   weights    (device) float [B][16 max_blocks], as lazy_attn_key_weights leaves them
 *   keep       (device) int32 [B]: document keys to keep; < 0 leaves the request's list as it is (nothing to
 *              move).  The first `first` and the last `recent` document keys go before all others, then the
 *              largest weights (NaN last); among equals the one that is earlier in the list.
 *   dst_pages  (device) int32 [B][max_dst]: pages for the kept keys, none of them in a list of this call.  A
 *              document with n kept keys takes ceil(n / 16) of them; keep / 16 + its number of documents
 *              always suffice.  Where they do not, or a page lies outside [0, num_pages), the status gets
 *              LAZY_STATUS_BAD_PAGE and the block's word is left without keys.
 *   new_meta   (device, written) uint64 [B][max_blocks]: the new list, kept keys first, then the query
 *              segment's blocks (all words from doc_blocks[b] on); the rest 0
 *   new_doc_blocks  (device, written) int32 [B];  seq_len and q_start stay valid
 *   src_slot, dst_slot  (device, written) int32 [B][16 max_dst]: rows to move (lazy_kv_move), -1 where none
 *   new_weights  (device, written) float [B][16 max_blocks]: the weights in the new list's order
 * A document is a run of blocks with one Delta.  meta and weights are only read.
 */
int lazy_evict_plan(const float* weights, const uint64_t* meta, const int32_t* doc_blocks,
                    const int32_t* keep, int first, int recent, const int32_t* dst_pages, int max_dst, int B,
                    int max_blocks, int num_pages, const lazy_pos_cfg* cfg, uint64_t* new_meta,
                    int32_t* new_doc_blocks, int32_t* src_slot, int32_t* dst_slot, float* new_weights,
                    void* stream);

/*
 * lazy_kv_move -- copy T rows of the caches: keys and values of slot src_slot[i] to dst_slot[i], every head,
 * bit for bit (eviction, or a private copy of a page that several requests share).  Entries with a
 * negative source or destination are skipped; one outside the caches sets LAZY_STATUS_BAD_SLOT and is
 * skipped.  Destinations must be distinct, and none may be a source of the same call.
 */
int lazy_kv_move(const int32_t* src_slot, const int32_t* dst_slot, int T, int Hkv, int D, void* k_cache,
                 void* v_cache, int num_pages, void* stream);

#define LAZY_PHASE_DECODE 0
#define LAZY_PHASE_PREFILL 1
#define LAZY_PHASE_DECODE_Q4 2
#define LAZY_PHASE_PREFILL_Q4 3
#define LAZY_PHASE_KEY_WEIGHTS 4

/*
 * lazy_workspace_size -- bytes of workspace the given call needs (0 if none); phase is one of the
 * LAZY_PHASE_* above.  rows = B for decode, total_q for prefill and key weights.  Uses the current device's SM count, so query it
 * with the device that will run the call current.
 */
size_t lazy_workspace_size(int phase, int rows, int B, int max_blocks, int Hq, int Hkv, int D);

/*
 * lazy_device_status -- synchronise `stream`, then read and clear the current device's
 * status word into *status (LAZY_STATUS_* bits; 0 = no kernel reported a problem).
 */
int lazy_device_status(void* stream, uint32_t* status);

/* Thread-local message for the last non-zero return code of this thread. */
const char* lazy_last_error(void);

/* ------------------------------------------------------------------------------------------
 * Document cache manager (host only).  [NOTE] 研究背景与动机 (核心矛盾: with a Zipf document
 * popularity, D possible positions and a budget of C entries, a position-free cache holds the
 * top C documents while a position-aware one holds only floor(C/D) of them) and 关键设计
 * (Deferred Positional Encoding: one physical copy serves every position).
 * Decides which documents' pages are resident in a pool of num_pages pages ([0, num_pages) of
 * the K/V caches).  position_aware = 0: one entry per document (this library's cache);
 * position_aware = 1: one entry per (document, position) variant (the design the pages
 * compare against; for simulation).  Least-recently-used eviction among entries no batch
 * holds.  The handle is host memory owned by the caller (create / destroy); not thread-safe.
 * ------------------------------------------------------------------------------------------ */
typedef struct lazy_doc_cache lazy_doc_cache;
/* NULL on error (num_pages outside [1, 2^24]; lazy_last_error says why). */
lazy_doc_cache* lazy_doc_cache_create(int num_pages, int position_aware);
void lazy_doc_cache_destroy(lazy_doc_cache* cache);
/* Look up without changing recency or pins: returns the entry's page count (its page ids copied
 * to pages_out (host) if not NULL and max_pages is large enough), 0 if not resident, < 0 on an
 * argument error.  `pos` is ignored by a position-agnostic cache. */
int lazy_doc_cache_lookup(lazy_doc_cache* cache, int doc, int pos, int32_t* pages_out, int max_pages);
/* Hold document `doc` (at position `pos`) for a batch: on a hit (*hit = 1) copies its n_pages
 * page ids to pages_out (host); on a miss (*hit = 0) evicts unheld least-recently-used entries
 * until n_pages pages are free and assigns them (the caller then writes the document there, e.g.
 * with lazy_kv_write at local positions).  Either way the entry is pinned until
 * lazy_doc_cache_release.  LAZY_ERANGE if held entries leave no room; LAZY_EINVAL on bad
 * arguments or a cached entry of another size. */
int lazy_doc_cache_acquire(lazy_doc_cache* cache, int doc, int pos, int n_pages, int32_t* pages_out, int* hit);
int lazy_doc_cache_release(lazy_doc_cache* cache, int doc, int pos);
/* Counters since creation (any pointer may be NULL). */
int lazy_doc_cache_stats(const lazy_doc_cache* cache, long long* hits, long long* misses, long long* evictions,
                         int* entries, int* free_pages);

/* Library version, e.g. 100 for 0.1.0. */
int lazy_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LAZYKV_H */
