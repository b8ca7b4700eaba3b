/*
 * hsa.h -- C ABI of the Hybrid-SWA dual-KV-pool attention library (libhsa.so).
 *
 * The model interleaves sliding-window layers (window W = 128) with full-attention
 * layers (60 : 10 in a 70-layer stack, 6:1).  Full layers keep every token in a
 * paged Full KV Pool that grows on demand; sliding layers keep only the last W
 * tokens of each sequence in a ring-buffer SWA KV Pool (slot = pos mod W), so
 * their storage is O(W).  One unified sequence view: the block table (full index)
 * is authoritative, and the ring row is the mapping into the SWA pool.
 * Sources: youleyou.com "小米MiMo首次公开模型推理系统全链路优化降价99%", s1
 * "为什么选择 Hybrid SWA 架构" and s2 "KVCache系统重构"; hotdry.top "MiMo-V2.5
 * ultra-speed inference architecture", "Hybrid SWA" and "三层 KVCache 系统".
 *
 * Conventions shared by every entry point
 *  - All tensors are caller-owned DEVICE memory unless a parameter says "host".
 *    The library never allocates, frees or synchronises; every kernel is queued on
 *    `stream` (a cudaStream_t; NULL = legacy default stream) and the call returns
 *    once it is queued.
 *  - bf16 tensors are little-endian IEEE bfloat16, densely packed, row-major, with
 *    the shapes given below; every device pointer must be 16-byte aligned.
 *  - Host-detectable errors are returned synchronously and nothing is launched.
 *    Range errors that only the device can see (a block-table entry outside the
 *    pool, a position past the block table, a ring row outside the ring) are
 *    OR-ed into *dev_err (device int32, caller zeroes it) as HSA_DEVERR_* bits;
 *    the offending item is skipped or its keys treated as absent, never trapped.
 *  - Attention calls never modify the pools; only the appends do (hsa_kv_append,
 *    hsa_rope_kv_append, and a decode call that is asked to append), and hsa_kv_compact.
 *  - Attention reads pool positions < cached/prefix length only; the current
 *    step's new tokens are read from k_new/v_new.  For several new tokens on a
 *    sliding layer (MTP verify, prefill chunks) call append AFTER attention:
 *    appending first would overwrite ring slots the earlier queries still need.
 *  - Query head h uses KV head h / (Hq / Hkv).  A sliding-window query at
 *    position p attends positions max(0, p-W+1) .. p (W keys including itself).
 *  - A call runs on the current device, which has to be its tensors' and its stream's.
 */
#ifndef HSA_H
#define HSA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int hsa_status;
#define HSA_OK 0
#define HSA_INVALID_ARG 1        /* null pointer, negative size, bad layer index */
#define HSA_UNSUPPORTED_SHAPE 2  /* head_dim != 128, page != 64, W not a multiple of 64, ... */
#define HSA_CUDA_ERROR 3         /* a CUDA runtime call failed (launch, attribute, ...) */
#define HSA_OUT_OF_RANGE 4       /* a caller buffer is too small for the result (host calls) */

/* bits OR-ed into *dev_err by the kernels */
#define HSA_DEVERR_BAD_BLOCK 1   /* block-table entry outside [0, num_blocks) */
#define HSA_DEVERR_BAD_PAGE 2    /* position needs a logical page >= max_blocks */
#define HSA_DEVERR_BAD_SEQ 4     /* sequence index outside [0, batch) */
#define HSA_DEVERR_BAD_RING 8    /* ring row outside [0, n_ring_rows) */
#define HSA_DEVERR_BAD_LEN 16    /* negative length or offsets out of order */
#define HSA_DEVERR_TIMEOUT 32    /* a bounded wait inside a kernel (2 s) gave up: the kernel
                                    stopped early and its outputs are incomplete */

/* FP8 formats of a Full KV Pool layer (hsa_pools.layer_kv_fp8). */
#define HSA_KV_E4M3 1
#define HSA_KV_E5M2 2

/*
 * The dual KV pool of one model (host struct of device pointers).
 *  layer_is_full[l]  host uint8: 1 = full layer (Full KV Pool), 0 = sliding layer.
 *  k[l], v[l]        host arrays of device pointers, one K and one V tensor per layer:
 *                    full layer:    [num_blocks, Hkv, page_size, d] bf16
 *                                   (a block holds page_size consecutive positions;
 *                                   each (block, head) tile is contiguous)
 *                    sliding layer: [n_ring_rows, Hkv, W, d] bf16, slot = pos mod W
 *  block_tables      device int32 [batch, max_blocks]: logical page -> physical block,
 *                    shared by every full layer; entries past a sequence's
 *                    allocation are never read.
 *  ring_row          device int32 [batch]: the SWA ring row of each sequence,
 *                    shared by every sliding layer.
 *  layer_kv_fp8      host uint8 [n_layers] or NULL: HSA_KV_E4M3 (1) or HSA_KV_E5M2
 *                    (2) = this full layer is an FP8 Full KV Pool layer of that
 *                    format, 0 = bf16, any other value HSA_INVALID_ARG
 *                    [hotdry.top "MiMo inference optimization, edge deployment",
 *                    "KV Cache 量化策略的技术选型": FP8 KV (E4M3 / E5M2), quantisation
 *                    groups aligned to the window; "边缘部署的工程权衡与参数清单": the
 *                    newest 128 tokens at the original precision -- a sliding
 *                    layer's ring, which holds exactly those, stays bf16].  Then k[l]
 *                    and v[l] each point to num_blocks * Hkv * 64 * (d + 4) bytes:
 *                    FP8 codes, then one fp32 scale per (block, head, row):
 *                      codes  [num_blocks * Hkv * 64 * d] bytes, then
 *                      scales [num_blocks * Hkv * 64] fp32, index (block*Hkv + h)*64 + row
 *                    K codes: page (block, h) = 64 rows of d bytes; dimension c of a
 *                    row at byte 16*(c/16) + perm16(c%16).  V codes (transposed):
 *                    page (block, h) = d rows of 64 bytes; key row r of dimension c at
 *                    byte 16*(r/16) + perm16(r%16) of row c.
 *                    perm16(l) = 4*((l%8)/2) + (l%2) + 2*(l/8).
 *                    scale = amax / F of the row's d values (fp32 division), F = 448
 *                    (E4M3) or 57344 (E5M2), the format's largest finite magnitude;
 *                    code = FP8 of value / scale (round to nearest even, saturating);
 *                    an all-zero row stores scale 0.  hsa_kv_append and
 *                    hsa_decode_attn_append quantise on write; decode reads such
 *                    layers; prefill rejects them (HSA_UNSUPPORTED_SHAPE), as does a
 *                    sliding layer flagged FP8.  Decode multiplies in fp16 there:
 *                    q, the new rows and |v| * 256 / 448 (E4M3) or |v| * 256 / 57344
 *                    (E5M2) must stay within fp16 range (hsa_decode_attn_weights: q
 *                    alone).
 * Supported shape: d = 128, page_size = 64, W a multiple of 64 in [64, 256],
 * Hq a multiple of Hkv with Hq / Hkv in {1, 2, 4, 8}.
 */
typedef struct hsa_pools {
    int32_t n_layers;
    const uint8_t *layer_is_full;
    void *const *k;
    void *const *v;
    int32_t num_blocks;
    int32_t page_size;
    const int32_t *block_tables;
    int32_t max_blocks;
    const int32_t *ring_row;
    int32_t n_ring_rows;
    int32_t batch;
    int32_t W;
    int32_t Hq;
    int32_t Hkv;
    int32_t d;
    const uint8_t *layer_kv_fp8;
} hsa_pools;

/*
 * KV append [youleyou s2 "KVCache系统重构": Full KV Pool grows on demand; SWA KV
 * Pool is a ring buffer of W slots per sequence].
 * Request r appends rows cu_tokens[r] .. cu_tokens[r+1]-1 of k_new / v_new
 * ([ntok, Hkv, d] bf16) to sequence seq_idx[r] at positions start_pos[r] + i.
 *  full layer:    K/V row -> pool[block_tables[seq][pos / page]][h][pos % page]
 *  sliding layer: K/V row -> ring[ring_row[seq]][h][pos % W]; of a request longer
 *                 than W only its last W tokens are written (each slot once),
 *                 which equals appending every token in position order.
 * cu_tokens, seq_idx, start_pos are device int32 arrays; cu_tokens[R] == ntok.
 * A sequence may appear in at most one request per call.
 */
hsa_status hsa_kv_append(const hsa_pools *pools, int32_t layer, const void *k_new,
                         const void *v_new, const int32_t *cu_tokens, const int32_t *seq_idx,
                         const int32_t *start_pos, int32_t R, int32_t ntok,
                         int32_t *dev_err, void *stream);

/*
 * Rotary positions.  Token n's position on axis a is positions[a * n_tokens + n]; pair i of a
 * head's first rot_dim values, (x[i], x[i + rot_dim / 2]) or, interleaved, (x[2i],
 * x[2i + 1]), is turned by the angle t = position on axis axis_of_pair[i] * inv_freq[i]:
 *   (x, y) -> scale * (x cos t - y sin t, y cos t + x sin t)
 * Values past rot_dim pass unchanged (not scaled).  Text has one axis; an image's or a
 * video's tokens have several (time, height, width), each with a section of the pairs.
 * Whole turns are taken off to within 2^-31 of a turn at every int32 position (not by an
 * fp32 product); the rest is rounded to fp32, 2^-26 of a turn at most, and the rotation is
 * fp32, rounded once to bf16.  Positions may be negative: negated positions undo a rotation
 * (scale 1).
 *  rot_dim       a multiple of 16 in [16, d] (else HSA_UNSUPPORTED_SHAPE)
 *  n_axes        1 .. 4
 *  interleaved   0: pairs (i, i + rot_dim / 2); 1: pairs (2i, 2i + 1)
 *  scale         of the turned values (1, or a context extension's attention factor)
 *  inv_freq      host double [rot_dim / 2]; finite
 *  axis_of_pair  host uint8 [rot_dim / 2], each < n_axes, or NULL: every pair on axis 0
 * The host arrays are read during the call only.
 */
typedef struct hsa_rope_params {
    int32_t rot_dim;
    int32_t n_axes;
    int32_t interleaved;
    float scale;
    const double *inv_freq;
    const uint8_t *axis_of_pair;
} hsa_rope_params;

/*
 * Turns the query and key heads of n tokens.  Before attention with several new tokens on
 * a sliding layer (MTP verify, prefill chunks), where the append has to come after it;
 * otherwise hsa_rope_kv_append does both in one launch.
 *  q  [n, Hq, d] bf16, k [n, Hkv, d] bf16: the heads of a token are contiguous, tokens are
 *     q_stride / k_stride elements apart (0 = dense; else a multiple of 8, at least one
 *     token's heads, at most 2^31), so slices of a QKV projection's rows serve.
 *  q_out, k_out  dense; q_out may be q itself and k_out k itself when those are dense, and
 *     must not overlap an input or each other otherwise (HSA_INVALID_ARG).
 *  positions     device int32 [n_axes, n]
 * Hq = 0 or Hkv = 0 leaves that side out (its pointers may be NULL).  d = 128.
 */
hsa_status hsa_rope(const hsa_rope_params *rope, const void *q, int64_t q_stride, const void *k,
                    int64_t k_stride, const int32_t *positions, int32_t n, int32_t Hq, int32_t Hkv,
                    int32_t d, void *q_out, void *k_out, void *stream);

/*
 * hsa_kv_append with the rotation on the way: the keys are turned, then keys and values
 * are written where hsa_kv_append would write them (same requests, same pool rows, same
 * dev_err bits), and the query heads are turned beside them.  Any layer: full (bf16 or
 * FP8) or sliding.
 *  q, k_new, v_new  as hsa_rope's q and k, with strides of their own.  q and q_out may
 *     both be NULL (keys alone).
 *  q_out            [ntok, Hq, d]: the turned queries
 *  k_out            [ntok, Hkv, d] or NULL: the turned keys, for the attention calls
 *  positions        device int32 [n_axes, ntok], or NULL: a token's cache position
 *                   (start_pos[r] + i) on every axis
 * An FP8 layer quantises the turned fp32 values (one rounding); hsa_rope followed by
 * hsa_kv_append would round them to bf16 first.  bf16 pools get the same bits either way.
 * A token of no request, or at a negative cache position, is skipped whole and flagged
 * (HSA_DEVERR_BAD_LEN): its rows of q_out and k_out stay as they were.  A token whose
 * pool row cannot be reached is flagged and not appended, but its q_out and k_out rows are
 * written.  ntok = 0 or R = 0: nothing is done.  On a sliding layer with several new tokens
 * append only after attention.
 */
hsa_status hsa_rope_kv_append(const hsa_pools *pools, int32_t layer, const hsa_rope_params *rope,
                              const void *q, int64_t q_stride, const void *k_new,
                              int64_t k_stride, const void *v_new, int64_t v_stride,
                              const int32_t *positions, const int32_t *cu_tokens,
                              const int32_t *seq_idx, const int32_t *start_pos, int32_t R,
                              int32_t ntok, void *q_out, void *k_out, int32_t *dev_err,
                              void *stream);

/*
 * Decode / MTP-verify attention [youleyou s1: decode latency tracks the KV bytes
 * read; s2 "Decode加速与多模态优化": 3-layer MTP, several candidate tokens verified
 * per step].  Sequence b (row b of block_tables / ring_row) has cached_len[b]
 * tokens in the pools and T new tokens at positions cached_len[b] + t, causal
 * among themselves.
 *  q      [B, T, Hq, d] bf16      k_new, v_new [B, T, Hkv, d] bf16
 *  out    [B, T, Hq, d] bf16      cached_len   device int32 [B]
 *  T in 1..4 (else HSA_UNSUPPORTED_SHAPE).  Full layers attend positions 0 .. cached_len+t; sliding layers
 *  attend the last W positions, the cached part read from the ring.
 *  Full layers split each sequence's pages across all SMs (flash-decoding) and
 *  merge the partial softmax states in the same kernel; that needs `workspace`
 *  of at least hsa_decode_workspace_bytes() bytes, ZERO-FILLED ONCE after
 *  allocation (every call leaves its arrival counters, at the start, zeroed again; the
 *  rest may hold anything).  The counters have room for pools->batch sequences, so one
 *  workspace serves calls of any B up to the one it was sized for, in any order, on any
 *  pools with the same batch and Hkv.  Calls sharing one workspace must not run
 *  concurrently.  After a call that set any bit in *dev_err, zero the workspace again
 *  before reusing it.
 *  max_ctas: 0 = one persistent CTA per SM (the default); > 0 caps the CTA count
 *  (results do not depend on it beyond rounding).
 */
size_t hsa_decode_workspace_bytes(const hsa_pools *pools, int32_t B, int32_t T);

hsa_status hsa_decode_attn(const hsa_pools *pools, int32_t layer, const void *q,
                           const void *k_new, const void *v_new, const int32_t *cached_len,
                           int32_t B, int32_t T, float scale, void *out, void *workspace,
                           size_t ws_bytes, int32_t max_ctas, int32_t *dev_err, void *stream);

/*
 * Decode attention fused with the append of the step's new tokens (the usual
 * decode step: attend, then keep the new K/V).  Same arguments and outputs as
 * hsa_decode_attn; in addition the T new rows of every sequence are written to
 * this layer's pool at positions cached_len[b] + t (Full KV Pool page through the
 * block table, or ring slot (cached_len[b] + t) mod W), exactly what hsa_kv_append
 * with one request per sequence would write.  Each (sequence, KV head) is appended
 * by the CTA that finishes its attention, after every read of it, so T > 1 on a
 * sliding layer is safe.  For MTP verify where only some drafts are accepted, use
 * hsa_decode_attn and then hsa_kv_append with the accepted tokens instead.
 */
hsa_status hsa_decode_attn_append(const hsa_pools *pools, int32_t layer, const void *q,
                                  const void *k_new, const void *v_new,
                                  const int32_t *cached_len, int32_t B, int32_t T, float scale,
                                  void *out, void *workspace, size_t ws_bytes, int32_t max_ctas,
                                  int32_t *dev_err, void *stream);

/*
 * Decode attention with options (a bit mask; other bits give HSA_INVALID_ARG):
 *  HSA_DECODE_APPEND           append the new rows as hsa_decode_attn_append does.
 *  HSA_DECODE_EARLY_POOL_READ  sliding layers: the kernel starts reading cached_len,
 *      ring_row and this layer's ring before the kernel queued just before it on
 *      `stream` has finished.  The decode kernels are launched with programmatic
 *      dependent launch: they may start once the previous kernel signals its
 *      dependents (this library's decode kernels signal at their start), and they
 *      read q, k_new, v_new and write out / the pools only after it has completed.
 *      With this option the caller guarantees that the kernel just before does not
 *      write cached_len, ring_row or this layer's ring: in a model that kernel is the
 *      layer's QKV projection (it writes q, k_new, v_new only); in a run of decode
 *      calls layer after layer it is the previous layer's attention.  A kernel that
 *      does not signal its dependents early (hsa_kv_append, for one) has completed
 *      before this one starts, so it may write anything.  The option lets the next
 *      layer's ring loads overlap the current layer's kernel (two sliding-layer CTAs
 *      fit on an SM for T <= 2).  Results are those of the same call without it.
 *      Full layers ignore it.
 * Same arguments and results as hsa_decode_attn otherwise.
 */
#define HSA_DECODE_APPEND 1
#define HSA_DECODE_EARLY_POOL_READ 2
hsa_status hsa_decode_attn_ex(const hsa_pools *pools, int32_t layer, const void *q,
                              const void *k_new, const void *v_new, const int32_t *cached_len,
                              int32_t B, int32_t T, float scale, void *out, void *workspace,
                              size_t ws_bytes, int32_t max_ctas, int32_t options,
                              int32_t *dev_err, void *stream);

/*
 * Decode / MTP-verify attention of a batch whose groups of sequences share their first
 * pages (a system prompt, a document, several samples of one prompt: what the prefix tree
 * hands out).  Same results as hsa_decode_attn_ex, beyond rounding; on a bf16 full layer
 * the shared pages are read once for a group instead of once for each sequence.  Rounding:
 * over shared pages a row's sum takes weights that the products round to bf16, so a row whose
 * weight is on few keys may be off by a further 2^-8 of itself.  Range: weights reach 2^16
 * between two updates of a row's maximum (2^8 in hsa_decode_attn_ex), so a value times the
 * number of keys has to stay below 2^111.
 *  cu_group    device int32 [n_groups + 1], 0 = cu_group[0] <= ... <= cu_group[n_groups]
 *              = B: group g is sequences cu_group[g] .. cu_group[g + 1] - 1
 *  shared_len  device int32 [n_groups]: tokens whose pages the group shares (>= 0).  Their
 *              whole pages, shared_len[g] / 64, have to be the same block-table entries in
 *              every row of the group as far as that member's cached tokens go; a part of a
 *              page is each sequence's own.  A member may have fewer cached tokens than
 *              shared_len (it sees its own), but must not append then: its new rows would
 *              land in a shared page.  The pages are read through the first member's row and
 *              shared as far as its cached tokens go, the others' further ones as their own:
 *              put a member that holds them all first.  Values of the shared pages have to be
 *              finite, also for a member that does not see them (it multiplies them by 0).
 *  n_groups    0 is hsa_decode_attn_ex.  Groups may be empty or of one sequence.
 *  options     as in hsa_decode_attn_ex.  The appended rows go to each sequence's own pages.
 *  workspace   at least hsa_decode_shared_workspace_bytes() bytes, with the rules of
 *              hsa_decode_attn's; it serves calls of fewer sequences, tokens and groups, and
 *              hsa_decode_attn_ex's, in any order.
 *  scale       > 0
 * Offsets out of order are flagged (HSA_DEVERR_BAD_LEN) and nothing is shared then: every
 * sequence reads its own pages, with the same results.  A negative shared_len is flagged and
 * taken as 0, one past the block table (HSA_DEVERR_BAD_PAGE) as its width.  Sliding layers
 * (a ring is its sequence's own) and FP8 layers run hsa_decode_attn_ex, as do block tables
 * with room for 2^31 half pages and more over all sequences and KV heads.
 */
size_t hsa_decode_shared_workspace_bytes(const hsa_pools *pools, int32_t B, int32_t T,
                                         int32_t n_groups);

hsa_status hsa_decode_attn_shared(const hsa_pools *pools, int32_t layer, const void *q,
                                  const void *k_new, const void *v_new,
                                  const int32_t *cached_len, const int32_t *cu_group,
                                  const int32_t *shared_len, int32_t n_groups, int32_t B,
                                  int32_t T, float scale, void *out, void *workspace,
                                  size_t ws_bytes, int32_t max_ctas, int32_t options,
                                  int32_t *dev_err, void *stream);

/*
 * hsa_decode_attn without a caller workspace.  The pages have no counterpart: this
 * is a convenience of this library for callers that cannot allocate device memory
 * where they run decode (while a stream is being captured, inside a host runtime
 * that owns every allocation, or in a loop that must never wait on cudaMalloc).
 * Same arguments and results as hsa_decode_attn minus `workspace` / `ws_bytes`.
 * The scratch is a fixed 8 MiB device array inside libhsa, held by every GPU that
 * loads the library until the process exits; it covers any batch with
 * B * Hkv <= 4096 (larger returns HSA_UNSUPPORTED_SHAPE) and caps the CTA count
 * at what fits (about 250).  This call allocates and frees nothing.
 *  - The first call on a device looks up the array's device address (and may load
 *    the library's device code): make that first call before any stream capture.
 *    The address is kept until the process exits: do not call this again after
 *    cudaDeviceReset (or another teardown of the device's primary context).
 *  - Each call zeroes the counter part of the array on `stream`, then launches.
 *  - All calls share the one array, so calls whose kernels could overlap on the
 *    GPU (different streams, or different host threads) race; serialise them.
 */
hsa_status hsa_decode_attn_noalloc(const hsa_pools *pools, int32_t layer, const void *q,
                                   const void *k_new, const void *v_new,
                                   const int32_t *cached_len, int32_t B, int32_t T, float scale,
                                   void *out, int32_t max_ctas, int32_t *dev_err, void *stream);

/*
 * Chunked prefill on a cached prefix [youleyou s1: SWA cuts prefill compute to
 * the window; hotdry.top "PD 分离与长度分桶": chunked prefill].
 * Request r has prefix_len[r] tokens in the pools of sequence seq_idx[r] and new
 * rows cu_rows[r] .. cu_rows[r+1]-1 at positions prefix_len[r] + i.
 *  q  [rows, Hq, d] bf16     k_new, v_new [rows, Hkv, d] bf16    out [rows, Hq, d] bf16
 *  cu_rows [R+1], prefix_len [R], seq_idx [R]: device int32.
 *  max_chunk: host upper bound on any request's row count (sizes the grid); rows of a
 *  request past the bound it implies are left unwritten, so it must not understate.
 * A sliding layer needs the ring to hold the prefix's last W positions.
 */
hsa_status hsa_prefill_attn(const hsa_pools *pools, int32_t layer, const void *q,
                            const void *k_new, const void *v_new, const int32_t *cu_rows,
                            const int32_t *prefix_len, const int32_t *seq_idx, int32_t R,
                            int32_t rows, int32_t max_chunk, float scale, void *out,
                            int32_t *dev_err, void *stream);

/*
 * Eviction from a full layer by accumulated attention weight (the pages have no counterpart:
 * their full layers keep every token).  A sliding layer's ring evicts by position alone; a
 * full layer grows with its sequence, and these calls bound it: hsa_prefill_weights and
 * hsa_decode_attn_weights sum the softmax weight that each cached key gets, hsa_kv_select
 * chooses the positions of a budget, and hsa_kv_compact moves their rows to pages of their
 * own, after which the full layers go on as those of a sequence of that many cached tokens.
 *
 * From then on a sequence has two lengths.  Calls on a full layer take new_len plus the tokens
 * since.  Calls on a sliding layer take the number of all its tokens, as if nothing had been
 * evicted, and so do hsa_window_safe_len and the rotary positions (`positions` of hsa_rope and
 * hsa_rope_kv_append; keys keep the rotation they were appended with).  A ring's slots and
 * window go by position: given the shorter length, the attention reads the wrong keys and the
 * append overwrites slots that are still seen, and nothing flags it.  All full layers of a model
 * share one block table and so one length: they are evicted together, each by its own weights.
 * A page of an evicted sequence no longer holds 64 consecutive positions: give a prefix tree its
 * pages before.
 *
 * Weights are fp32 rows w[sequence][KV head][w_stride], one value a cache position, w_stride a
 * multiple of 4, at most 2^30 (else HSA_INVALID_ARG).  An entry is the sum over the queries t and
 * the query heads of the KV head of exp(scale q.k - lse), lse the query's log of the sum over
 * every key that it sees.  Both calls write w[j] = decay * w_prev[j] + sum; w_prev (same layout)
 * may be w itself, or NULL: nothing before.  Positions that are new in the call count nothing from
 * w_prev.  Entries past a sequence's tokens are left as they were.  Sums are fp32, in an
 * order that does not change from call to call.
 */

/*
 * Decode / MTP-verify attention that also weighs the cached keys.  Arguments and output as
 * hsa_decode_attn_ex's on a full layer, bf16 or FP8 (a sliding layer: HSA_UNSUPPORTED_SHAPE);
 * sequence b's weights are row b of w, its new tokens' at cached_len[b] + t.
 *  decay      finite
 *  w_stride   cached_len[b] + T have to fit: a sequence whose tokens do not is flagged
 *             (HSA_DEVERR_BAD_LEN) and left out, its rows of out and w as they were, and not
 *             appended
 *  workspace  at least hsa_decode_weights_workspace_bytes() bytes for this B, T and w_stride;
 *             its contents do not matter before or after (0 bytes: a shape that the call
 *             refuses).  It holds every score in fp32:
 *             4 * T * Hq * B * w_stride bytes (T and Hq / Hkv's product rounded up to a
 *             power of two, at least 2) and the partial states.  Calls sharing one must
 *             not run concurrently.
 *  max_ctas   as in hsa_decode_attn, of each of the two launches
 *  options    HSA_DECODE_APPEND (other bits: HSA_INVALID_ARG)
 *  scale      2^-96 .. 2^96 (else HSA_INVALID_ARG)
 * A key whose page cannot be read is absent (flagged as in hsa_decode_attn): its weight is 0.
 * With T > 1 all T queries weigh, those of drafts that are rejected later among them, and a sum
 * cannot be taken apart again.  Where they should not count, let w be another buffer than w_prev,
 * and call again from the same w_prev with the accepted tokens alone (that call can append them).
 */
size_t hsa_decode_weights_workspace_bytes(const hsa_pools *pools, int32_t B, int32_t T,
                                          int32_t w_stride);

hsa_status hsa_decode_attn_weights(const hsa_pools *pools, int32_t layer, const void *q,
                                   const void *k_new, const void *v_new,
                                   const int32_t *cached_len, int32_t B, int32_t T, float scale,
                                   void *out, const float *w_prev, float decay, float *w,
                                   int32_t w_stride, void *workspace, size_t ws_bytes,
                                   int32_t max_ctas, int32_t options, int32_t *dev_err,
                                   void *stream);

/*
 * The weight that a prompt's last queries put on every cached key.  Called after the append:
 * request r is sequence seq_idx[r] with kv_len[r] tokens in the pool, the newest of them rows
 * cu_rows[r] .. cu_rows[r+1]-1 of q ([rows, Hq, d] bf16, as given to hsa_prefill_attn); the
 * last min(window, number of rows) of those weigh, row i of n rows seeing the positions up to
 * kv_len[r] - n + i.  The weights are row seq_idx[r] of w ([pools->batch, Hkv, w_stride]).
 *  window     1 .. 64 (else HSA_UNSUPPORTED_SHAPE)
 *  workspace  at least hsa_prefill_weights_workspace_bytes(); as above
 *  decay finite, scale 2^-96 .. 2^96 (else HSA_INVALID_ARG), scores scale q.k below 2^30
 * bf16 full layers (a sliding or FP8 layer: HSA_UNSUPPORTED_SHAPE, as prefill itself refuses
 * FP8; an FP8 layer's prompt is weighed by hsa_decode_attn_weights of its last tokens).  A sequence may appear in at most one request per call.  A request without rows is left
 * out.  So is one that is flagged: offsets out of order or past `rows`, more rows than
 * kv_len[r], kv_len[r] negative or past w_stride (HSA_DEVERR_BAD_LEN), a bad sequence
 * (HSA_DEVERR_BAD_SEQ).  A key whose page cannot be read is flagged and absent.
 */
size_t hsa_prefill_weights_workspace_bytes(const hsa_pools *pools, int32_t R, int32_t window);

hsa_status hsa_prefill_weights(const hsa_pools *pools, int32_t layer, const void *q,
                               const int32_t *cu_rows, const int32_t *kv_len,
                               const int32_t *seq_idx, int32_t R, int32_t rows, int32_t window,
                               float scale, const float *w_prev, float decay, float *w,
                               int32_t w_stride, void *workspace, size_t ws_bytes,
                               int32_t *dev_err, void *stream);

/*
 * The positions that stay.  Request r is row seq_idx[r] of w ([batch, heads, w_stride]), with
 * kv_len[r] positions; w_stride at most 2^22 (else HSA_UNSUPPORTED_SHAPE).  For each of the
 * `heads` rows, of n > budget positions stay the first `sinks`, the last `recent` (sinks +
 * recent <= budget) and, of the others, those of the largest score until the budget is full: a
 * position's score is the largest weight among itself and its `reach` neighbours on each side
 * (0 .. 7), NaN counting as -infinity and -0 as 0; of equal scores the lowest position.  Of n <=
 * budget positions all stay.
 *  keep     int32 [R, heads, budget]: the positions, ascending; -1 past new_len[r]
 *  new_len  int32 [R]: min(kv_len[r], budget); must overlap neither kv_len nor seq_idx (HSA_INVALID_ARG)
 * heads is Hkv where every KV head keeps its own, or 1 for weights that the caller has summed.
 * kv_len[r] outside 0 .. w_stride (HSA_DEVERR_BAD_LEN) and a bad sequence (HSA_DEVERR_BAD_SEQ)
 * are flagged: nothing stays of them (new_len 0).
 */
hsa_status hsa_kv_select(const float *w, int32_t w_stride, int32_t batch, int32_t heads,
                         const int32_t *kv_len, const int32_t *seq_idx, int32_t R,
                         int32_t budget, int32_t sinks, int32_t recent, int32_t reach,
                         int32_t *keep, int32_t *new_len, int32_t *dev_err, void *stream);

/*
 * Moves the rows that stay.  For request r and each KV head h, the K and V rows of sequence
 * seq_idx[r] (through block_tables) at positions keep[r][h][i], i < new_len[r], are copied to
 * position i of the pages dst_tables[r] ([R, dst_blocks] int32, physical blocks); an FP8
 * layer's codes and scales as they are.  Any full layer (a sliding one:
 * HSA_UNSUPPORTED_SHAPE).  The destination pages are the caller's to hand out, and no request
 * of the call may read or write them otherwise: a sequence's old pages, which other sequences
 * may share, stay as they were.  Once every full layer is compacted, the destination pages
 * become the sequence's row of the block table and new_len[r] its cached tokens in the full
 * layers (sliding layers keep theirs, above).
 *  keep     int32 [R, heads, budget] as hsa_kv_select gives them, heads = Hkv or 1 (one
 *           list for every head; else HSA_UNSUPPORTED_SHAPE)
 *  w, w_dst [batch, Hkv, w_stride] or both NULL: the weights moved along, w_dst[seq][h][i] =
 *           w[seq][h][keep[r][h][i]]; must not overlap.  With them a sequence may appear in
 *           one request per call; without, it may be moved to the pages of several
 * Rows of a destination page at new_len[r] and past it are left as they were.  Flagged, and
 * not copied: a position outside the block table (HSA_DEVERR_BAD_PAGE; a negative one, or
 * new_len[r] outside 0 .. budget, HSA_DEVERR_BAD_LEN), a bad block on either side
 * (HSA_DEVERR_BAD_BLOCK), a destination past dst_blocks (HSA_DEVERR_BAD_PAGE), a bad sequence
 * (HSA_DEVERR_BAD_SEQ).  A weight is copied if its position and its place lie below w_stride.
 */
hsa_status hsa_kv_compact(const hsa_pools *pools, int32_t layer, const int32_t *keep,
                          int32_t heads, int32_t budget, const int32_t *new_len,
                          const int32_t *seq_idx, int32_t R, const int32_t *dst_tables,
                          int32_t dst_blocks, const float *w, float *w_dst, int32_t w_stride,
                          int32_t *dev_err, void *stream);

/*
 * Layerwise SWA-KV prefetch [youleyou s2 "KVCache系统重构": the SWA layers' KV is
 * prefetched layer by layer, overlapped with compute, so reading the cache costs
 * almost nothing; hotdry.top "三层 KVCache 系统": host-to-device KV loads overlap the
 * compute stream].  Copies ring rows of sliding layer `layer` from a host tier into
 * the device SWA KV Pool: entry i moves row host_row[i] of host_k / host_v
 * ([n_host_rows, Hkv, W, d] bf16 in PINNED host memory, which the GPU reads
 * directly) into ring row ring_row[seq_idx[i]] of the layer.
 *  host_row, seq_idx: device int32 [n].  Full layers are rejected (HSA_INVALID_ARG),
 *  as is host memory that is not pinned.  Launch it on a side stream ahead of the
 *  attention that reads the layer and order the two with an event.
 */
hsa_status hsa_swa_prefetch(const hsa_pools *pools, int32_t layer, const void *host_k,
                            const void *host_v, int32_t n_host_rows, const int32_t *host_row,
                            const int32_t *seq_idx, int32_t n, int32_t *dev_err, void *stream);

/*
 * Window-safe prefix length [youleyou s2 "KVCache系统重构": a prefix match counts
 * only while the last W tokens still hold valid SWA slots; hotdry.top "Hybrid
 * SWA": the match length is cut back to the window boundary].
 * out_len[k] = the largest L in [0, match_len[k]] such that every position in
 * [max(0, L-W), L) is live.  The full-pool KV is taken as live on [0, match_len).
 *  ring form:   swa_slot_pos [n, W] device int32, the position each ring slot holds
 *               (-1 = freed); position p is live iff swa_slot_pos[p mod W] == p.
 *  bitmap form: live [live_off[n]] device uint8, live_off [n+1] device int64;
 *               position p of case k is live iff live[live_off[k] + p] != 0.
 * match_len, out_len: device int32 [n].  Negative match_len gives 0.
 */
hsa_status hsa_window_safe_len(const int32_t *match_len, const int32_t *swa_slot_pos,
                               int32_t n, int32_t W, int32_t *out_len, void *stream);

hsa_status hsa_window_safe_len_bitmap(const int32_t *match_len, const int64_t *live_off,
                                      const uint8_t *live, int32_t n, int32_t W,
                                      int32_t *out_len, void *stream);

/* Human-readable name of a status code (static string). */
const char *hsa_status_string(hsa_status s);

#ifdef __cplusplus
}
#endif

#endif /* HSA_H */
