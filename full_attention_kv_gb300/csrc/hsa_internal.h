// hsa_internal.h -- launch interfaces between the C-ABI layer (api.cu) and the
// kernels.  Host/device shared structs only; no kernel code.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/hsa.h"

struct __nv_bfloat16;

namespace hsa {

// A kernel's opt-in to its dynamic shared memory, which the runtime keeps for each device: set
// at the kernel's first call on a device (it is not a stream operation, but later calls, the
// captured ones among them, then make none).  Host threads may meet here: both then set it.
class SmemOptIn {
    std::atomic<uint64_t> done{0};  // bit = device; devices past 63 set it at every call

public:
    template <typename Kernel>
    cudaError_t set(Kernel kern, size_t bytes)
    {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess)
            return e;
        const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t(1) << dev : 0;
        if (done.load(std::memory_order_acquire) & bit)
            return cudaSuccess;
        e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kern),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess)
            done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// The decode parameter struct is passed by value and kept at <= 128 bytes: on
// sm_103a the decode kernel measured 19% slower with the same code when this
// struct grew from 128 to 136 bytes (a different code generation of the hot loop).
struct DecodeParams {
    const __nv_bfloat16 *q;      // [B, T, Hq, d]
    const __nv_bfloat16 *k_new;  // [B, T, Hkv, d]
    const __nv_bfloat16 *v_new;
    const int32_t *cached_len;   // [B]
    const int32_t *block_tables; // [batch, max_blocks]
    const int32_t *ring_row;     // [batch]
    __nv_bfloat16 *out;          // [B, T, Hq, d]
    uint8_t *ws;                 // workspace: arrival counters, then partial softmax states
    int32_t *dev_err;
    uint4 *k_dst;                // this layer's K pool / ring (append only)
    uint4 *v_dst;
    int32_t max_blocks, num_blocks, n_ring_rows;
    int32_t B, Hkv, W;
    int16_t T, G;                // query tokens per sequence; query heads per KV head
    int32_t flags;               // kDecode* bits below
    float scale_log2;            // softmax scale * log2(e)
};
constexpr int32_t kDecodeRing = 1;    // sliding layer: read the SWA ring
constexpr int32_t kDecodeAppend = 2;  // append the T new rows (hsa_decode_attn_append)
constexpr int32_t kDecodeFp8 = 4;     // full layer stored as FP8 codes + scales (fp8_kv.cuh)
constexpr int32_t kDecodeEarly = 8;   // sliding layer: walk and load the ring before the
                                      // grid-dependency wait (HSA_DECODE_EARLY_POOL_READ)
constexpr int32_t kDecodeE5M2 = 16;   // with kDecodeFp8: the codes are E5M2 (else E4M3)
static_assert(sizeof(DecodeParams) <= 128, "keep the decode parameter struct <= 128 bytes");

// Bytes of the arrival counters of B sequences.  A workspace begins with room for those of
// the pools' whole batch (decode_counted), so that no call's states lie where another call,
// of more sequences, counts arrivals.  A kernel is handed the end of that room less its own
// batch's counters, and finds its partial states right behind them.
__host__ __device__ inline size_t decode_counter_bytes(int B, int Hkv)
{
    return ((size_t)B * Hkv * sizeof(int32_t) + 255) & ~size_t(255);
}

size_t decode_workspace_bytes(int num_sms, int counted, int Hkv);
inline int decode_counted(const hsa_pools *pools, int B)
{
    return pools->batch > B ? pools->batch : B;
}
// hsa_decode_attn_ex on a workspace that holds counters for `counted` >= B sequences
// (counted = 0: of the pools' batch).
hsa_status decode_attn(const hsa_pools *pools, int32_t layer, const void *q, const void *k_new,
                       const void *v_new, const int32_t *cached_len, int32_t B, int32_t T,
                       float scale, void *out, void *workspace, size_t ws_bytes, int32_t max_ctas,
                       int32_t *dev_err, void *stream, int32_t options, int32_t counted);
// Every host-side check of a decode call except the workspace's (api.cu); HSA_OK
// with *done = true means there is nothing to do (B = 0).
hsa_status decode_host_check(const hsa_pools *pools, int32_t layer, const void *q,
                             const void *k_new, const void *v_new, const int32_t *cached_len,
                             int32_t B, int32_t T, const void *out, int32_t max_ctas, bool *done);
cudaError_t launch_decode(const CUtensorMap &tmK, const CUtensorMap &tmV, const DecodeParams &p,
                          int ctas, cudaStream_t stream);

// Decode over shared prefixes (decode_shared.cu): what its parts leave the merge
// in the workspace.
struct SharedGroup {
    int32_t item0;               // first item of the group in part 1's item space
    int32_t unit0;               // units of the groups before it
    int32_t pairs, pages;        // 256-row units a KV head; shared pages (items a unit)
};
struct SharedPlan {
    int32_t N, C;                // part 1's items, and the CTAs they were cut over
    SharedGroup group[1];        // [n_groups]
};
struct OwnPlan {
    int32_t N, C;                // part 2's, and its streams
    int32_t before[1];           // [B]: own items (of one head) of the sequences before
};
struct SharedLayout {            // byte offsets in the workspace
    size_t plan, own_plan, slots, own, total;
};
struct SharedParams {
    DecodeParams d;
    const int32_t *cu_group;     // [n_groups + 1]
    const int32_t *shared_len;   // [n_groups]
    int64_t plan_off, own_plan_off, slot_off, own_off;
    int32_t n_groups;
};

SharedLayout shared_layout(size_t start, int ctas, int B, int T, int G, int Hkv, int n_groups);
// Whether the items of both parts, at the longest that the block table has room for, and the
// merge's rows and threads count to below 2^31.
bool shared_fits(const SharedParams &p);
// tmK, tmV: boxes of a page; tmK32, tmV32: of half a page
cudaError_t launch_shared(const CUtensorMap &tmK, const CUtensorMap &tmV, const CUtensorMap &tmQ,
                          const CUtensorMap &tmK32, const CUtensorMap &tmV32,
                          const SharedParams &p, int ctas, int sms, cudaStream_t stream);

struct AppendParams {
    const uint4 *k_new;          // [ntok, Hkv, d] as 16-byte chunks
    const uint4 *v_new;
    const int32_t *cu_tokens;    // [R+1]
    const int32_t *seq_idx;      // [R]
    const int32_t *start_pos;    // [R]
    uint4 *k_dst;                // layer's K pool / ring
    uint4 *v_dst;
    const int32_t *block_tables;
    const int32_t *ring_row;
    int32_t *dev_err;
    int32_t R, ntok, Hkv, chunks_per_row;  // chunks_per_row = d * 2 / 16
    int32_t batch, max_blocks, num_blocks, page_size, n_ring_rows, W;
    int32_t ring_mode;
    int32_t fp8;                 // full layer stored as FP8 codes + scales (fp8_kv.cuh):
                                 // 0 bf16, 1 E4M3, 2 E5M2
};

cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);

// Rotary positions (rope.cu).  Rows are counted in 16-byte chunks: a head is 16 of them.
struct RopeParams {
    const uint4 *q, *k, *v;      // n rows of heads; row strides below
    uint4 *q_out, *k_out;        // [n, Hq, d], [n, Hkv, d] dense (k_out may be null)
    int64_t q_stride, k_stride, v_stride;
    const int32_t *pos;          // [n_axes, n]; null: the cache position on every axis
    int32_t n, Hq, Hkv;
    int32_t rot16;               // rot_dim / 16
    int32_t interleaved;
    int32_t quads;               // head quads an item takes (set by launch_rope)
    float scale;
    uint32_t axis2[4];           // axis of pair i: two bits at 2 (i % 16) of word i / 16
    uint64_t turn[64];           // inv_freq / 2 pi as a 64-bit fraction of a turn
    // append only
    const int32_t *cu_tokens;    // [R+1]
    const int32_t *seq_idx;      // [R]
    const int32_t *start_pos;    // [R]
    uint4 *k_dst, *v_dst;        // the layer's pool / ring
    const int32_t *block_tables;
    const int32_t *ring_row;
    int32_t *dev_err;
    int32_t R, batch, max_blocks, num_blocks, n_ring_rows, W;
    int32_t ring_mode;
    int32_t fp8;                 // 0 bf16, 1 E4M3, 2 E5M2
    int32_t v_apart;             // FP8: the values as items of their own, 16 tokens of a KV
                                 // head each, ahead of the tokens (set by launch_rope)
};

cudaError_t launch_rope(RopeParams &p, bool append, int sms, cudaStream_t stream);

// Prefill keeps its larger by-value struct: promoted into registers (<= 128
// bytes) it raised the prefill kernel's spills from 76 to 252 bytes.
struct PrefillParams {
    const __nv_bfloat16 *q;      // [rows, Hq, d]
    const __nv_bfloat16 *k_new;  // [rows, Hkv, d]
    const __nv_bfloat16 *v_new;
    const int32_t *cu_rows;      // [R+1]
    const int32_t *prefix_len;   // [R]
    const int32_t *seq_idx;      // [R]
    const int32_t *block_tables;
    const int32_t *ring_row;
    __nv_bfloat16 *out;          // [rows, Hq, d]
    int32_t *dev_err;
    int32_t R, rows, Hq, Hkv, G, W;
    int32_t batch, max_blocks, num_blocks, n_ring_rows;
    int32_t ring_mode;
    int32_t tiles_per_req_bound; // host upper bound on the total number of 128-row tiles
    float scale_log2;
};

size_t prefill_smem_bytes();
cudaError_t launch_prefill(const CUtensorMap &tmPoolK, const CUtensorMap &tmPoolV,
                           const CUtensorMap &tmNewK, const CUtensorMap &tmNewV,
                           const CUtensorMap &tmQ, const PrefillParams &p, cudaStream_t stream);

// Sliding layers whose window and GQA group fit one key tile (W + 128 / G + 16 <=
// 160 keys: W = 64 or 128 at G = 8, W = 64 at G = 2 or 4) run the persistent
// sliding-window prefill kernel
// (prefill_swa.cu); other sliding shapes run prefill_kernel in ring mode.
bool prefill_swa_supported(int W, int G);
cudaError_t launch_prefill_swa(const CUtensorMap &tmQ, const CUtensorMap &tmNewK,
                               const CUtensorMap &tmNewV, const CUtensorMap &tmRingK,
                               const CUtensorMap &tmRingV, const PrefillParams &p, int sms,
                               cudaStream_t stream);

// Eviction by accumulated weight.
struct WeighParams {             // decode_weights.cu
    const __nv_bfloat16 *q;      // [B, T, Hq, d]
    const __nv_bfloat16 *k_new;  // [B, T, Hkv, d]
    const __nv_bfloat16 *v_new;
    const int32_t *cached_len;   // [B]
    const int32_t *block_tables; // [batch, max_blocks]
    __nv_bfloat16 *out;          // [B, T, Hq, d]
    const float *w_prev;         // [B, Hkv, w_stride] or null
    float *w;
    float *part;                 // workspace: partial states, slot by slot
    float *score;                // workspace: [B, Hkv, w_stride, srow] scores in log2 units
    int32_t *dev_err;
    uint4 *k_pool, *v_pool;      // this layer's pools (FP8 scales; the append)
    int32_t max_blocks, num_blocks, B, Hkv, w_stride;
    int32_t T, G, srow;          // srow: G T rounded up to a power of two, at least 2
    int32_t append, fp8;         // fp8: 0 bf16, 1 E4M3, 2 E5M2
    float scale_log2, decay;
};
struct WeighLayout {             // byte offsets in the workspace
    size_t part, score, total;
};
WeighLayout weigh_layout(int ctas, int B, int T, int G, int Hkv, int w_stride);
cudaError_t launch_weigh(const CUtensorMap &tmK, const CUtensorMap &tmV, const WeighParams &p,
                         int sms, int max_ctas, cudaStream_t stream);

struct PromptParams {            // prefill_weights.cu
    const int32_t *cu_rows;      // [R+1]
    const int32_t *kv_len;       // [R]
    const int32_t *seq_idx;      // [R]
    const int32_t *block_tables;
    const float *w_prev;         // [batch, Hkv, w_stride] or null
    float *w;
    float2 *part;                // workspace: (m, l) of each slot's rows
    int32_t *dev_err;
    int32_t R, rows, window, Hkv, G, batch, max_blocks, num_blocks, w_stride;
    float scale_log2, decay;
};
size_t prompt_workspace_bytes(int ctas, int R, int Hkv);
cudaError_t launch_prompt_weights(const CUtensorMap &tmK, const CUtensorMap &tmQ,
                                  const PromptParams &p, int ctas, cudaStream_t stream);

struct SelectParams {            // kv_select.cu
    const float *w;              // [batch, heads, w_stride]
    const int32_t *kv_len, *seq_idx;
    int32_t *keep, *new_len, *dev_err;
    int32_t w_stride, batch, heads, R, budget, sinks, recent, reach;
    int32_t held;                // keys a CTA keeps the high halves of (set by launch_select)
};
cudaError_t launch_select(SelectParams &p, int sms, cudaStream_t stream);

struct CompactParams {           // kv_compact.cu
    uint4 *k, *v;                // the layer's pools
    const int32_t *keep, *new_len, *seq_idx, *block_tables, *dst_tables;
    const float *w;
    float *w_dst;
    int32_t *dev_err;
    int32_t heads, budget, R, dst_blocks, w_stride;
    int32_t batch, max_blocks, num_blocks, Hkv, fp8;
};
cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream);

struct SwaPrefetchParams {
    const uint4 *host_k;         // pinned host ring rows [n_host_rows, Hkv, W, d] (device-visible)
    const uint4 *host_v;
    uint4 *dev_k;                // the layer's device ring [n_ring_rows, Hkv, W, d]
    uint4 *dev_v;
    const int32_t *host_row;     // [n]
    const int32_t *seq_idx;      // [n]
    const int32_t *ring_row;     // [batch]
    int32_t *dev_err;
    int32_t n, n_host_rows, n_ring_rows, batch, Hkv, W, chunks_per_row;
};

cudaError_t launch_swa_prefetch(const SwaPrefetchParams &p, cudaStream_t stream);

cudaError_t launch_window_safe_ring(const int32_t *match_len, const int32_t *slot_pos, int32_t n,
                                    int32_t W, int32_t *out, cudaStream_t stream);
cudaError_t launch_window_safe_bitmap(const int32_t *match_len, const int64_t *live_off,
                                      const uint8_t *live, int32_t n, int32_t W, int32_t *out,
                                      cudaStream_t stream);

}  // namespace hsa
