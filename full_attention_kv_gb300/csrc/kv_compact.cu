// kv_compact.cu -- the rows of a full layer that stay, moved into pages of their own (sm_103a).
//
// What it does: for request r, KV head h and i < new_len[r], the K and V rows (and the weight) at
// position keep[r][h][i] of the sequence go to position i of the pages dst_tables[r].  Stored
// values move as they are: bf16 rows, or an FP8 layer's codes and scales (fp8_kv.cuh).
//
// One CTA a destination page of a head.  Its 64 source rows are found first (keep, then the block
// table), then every 16-byte chunk is one thread's: 256 contiguous bytes a bf16 row, 128 an FP8 K
// row.  An FP8 layer's V is stored transposed (64 keys of a dimension side by side), so a single
// key is 128 bytes in as many sectors; the source pages are taken whole instead, one after another
// (positions ascend, so a page's keys are neighbours in the list): 8 KB into shared memory, the
// wanted bytes into the destination page's tile there, and the tile out in 16-byte stores.  A
// word of either tile lies rotated by half its dimension, so that the 32 dimensions of a warp meet
// 32 banks.
#include "fp8_kv.cuh"
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kThreads = 256;
constexpr int kPage = 64;

// Word `w` (0 .. 15) of dimension `dim` in a V tile in shared memory.
__device__ __forceinline__ int v_word(int dim, int w) { return dim * 16 + ((w + (dim >> 1)) & 15); }

// Byte of key `row` of a page in a V row.
__device__ __forceinline__ int v_byte(int row) { return 16 * (row >> 4) + perm16(row & 15); }

template <bool FP8>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p)
{
    __shared__ int64_t src[kPage];  // a head's row in the pool, or -1
    __shared__ uint32_t ok[2];      // bit i: row i is to be copied
    __shared__ uint32_t from[FP8 ? 128 * 16 : 1], to[FP8 ? 128 * 16 : 1];
    const int tid = threadIdx.x, lane = tid & 31;
    const int pages = (p.budget + kPage - 1) / kPage;
    const int page = blockIdx.x % pages;
    const int64_t rh = blockIdx.x / pages;
    const int h = (int)(rh % p.Hkv), r = (int)(rh / p.Hkv);
    grid_dependency_wait();
    grid_launch_dependents();

    const int n = __ldg(p.new_len + r), seq = __ldg(p.seq_idx + r);
    const bool first = tid == 0 && h == 0 && page == 0;
    if (n < 0 || n > p.budget) {
        if (first)
            set_err(p.dev_err, HSA_DEVERR_BAD_LEN);
        return;
    }
    if (page * kPage >= n)
        return;
    if (seq < 0 || seq >= p.batch) {
        if (first)
            set_err(p.dev_err, HSA_DEVERR_BAD_SEQ);
        return;
    }
    if (page >= p.dst_blocks) {
        if (tid == 0)
            set_err(p.dev_err, HSA_DEVERR_BAD_PAGE);
        return;
    }
    const int dst_blk = __ldg(p.dst_tables + (int64_t)r * p.dst_blocks + page);
    if (dst_blk < 0 || dst_blk >= p.num_blocks) {
        if (tid == 0)
            set_err(p.dev_err, HSA_DEVERR_BAD_BLOCK);
        return;
    }
    const int64_t dst_row = ((int64_t)dst_blk * p.Hkv + h) * kPage;
    if (tid < kPage) {
        const int i = page * kPage + tid;
        int64_t row = -1;
        if (i < n) {
            const int pos = __ldg(p.keep + ((int64_t)r * p.heads + (p.heads > 1 ? h : 0)) * p.budget + i);
            int err = 0;
            if (pos < 0) {
                err = HSA_DEVERR_BAD_LEN;
            } else if (pos / kPage >= p.max_blocks) {
                err = HSA_DEVERR_BAD_PAGE;
            } else {
                const int blk = __ldg(p.block_tables + (int64_t)seq * p.max_blocks + pos / kPage);
                if (blk < 0 || blk >= p.num_blocks)
                    err = HSA_DEVERR_BAD_BLOCK;
                else
                    row = ((int64_t)blk * p.Hkv + h) * kPage + pos % kPage;
            }
            if (err)
                set_err(p.dev_err, err);
            if (p.w && pos >= 0 && pos < p.w_stride && i < p.w_stride) {
                const int64_t at = ((int64_t)seq * p.Hkv + h) * p.w_stride;
                p.w_dst[at + i] = __ldg(p.w + at + pos);
            }
        }
        src[tid] = row;
        const uint32_t b = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0)
            ok[tid >> 5] = b;
    }
    __syncthreads();

    if constexpr (!FP8) {
        // 16 rows at a time, a 16-byte chunk a thread; K's and V's loads all in flight
        const int ch = tid & 15, r0 = tid >> 4;
        uint4 x[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t s = src[r0 + 16 * j];
            if (s >= 0) {
                x[2 * j] = __ldcs(p.k + s * 16 + ch);
                x[2 * j + 1] = __ldcs(p.v + s * 16 + ch);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t d = (dst_row + r0 + 16 * j) * 16 + ch;
            if (src[r0 + 16 * j] >= 0) {
                p.k[d] = x[2 * j];
                p.v[d] = x[2 * j + 1];
            }
        }
    } else {
        const int64_t cb = fp8_codes_bytes(p.num_blocks, p.Hkv);
        float *const ks = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.k) + cb);
        float *const vs = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(p.v) + cb);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = (tid >> 3) + 32 * j;
            if (src[i] >= 0)
                p.k[(dst_row + i) * 8 + (tid & 7)] = __ldcs(p.k + src[i] * 8 + (tid & 7));
        }
        if (tid < kPage && src[tid] >= 0) {
            ks[dst_row + tid] = ks[src[tid]];
            vs[dst_row + tid] = vs[src[tid]];
        }
        // V: source pages in runs of the list
        const int dim = tid & 127, half = tid >> 7;
        const uint8_t *const fb = reinterpret_cast<const uint8_t *>(from);
        uint8_t *const tb = reinterpret_cast<uint8_t *>(to);
        int i = 0;
        while (i < kPage) {
            if (src[i] < 0) {  // the same for every thread
                ++i;
                continue;
            }
            const int64_t pg = src[i] / kPage;
            int end = i + 1;
            while (end < kPage && src[end] >= 0 && src[end] / kPage == pg)
                ++end;
            __syncthreads();  // `from` is free again
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = tid + kThreads * j;  // chunk e % 4 of dimension e / 4
                const uint4 x = __ldcs(p.v + pg * 512 + e);
                const int d = e >> 2, w = 4 * (e & 3);
                from[v_word(d, w)] = x.x;
                from[v_word(d, w + 1)] = x.y;
                from[v_word(d, w + 2)] = x.z;
                from[v_word(d, w + 3)] = x.w;
            }
            __syncthreads();
            for (int k = i + half; k < end; k += 2) {
                const int a = v_byte((int)(src[k] % kPage)), b = v_byte(k);
                tb[4 * v_word(dim, b >> 2) + (b & 3)] = fb[4 * v_word(dim, a >> 2) + (a & 3)];
            }
            i = end;
        }
        __syncthreads();
        const uint64_t have = (uint64_t)ok[1] << 32 | ok[0];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = tid + kThreads * j, d = e >> 2, g = e & 3;  // 16 keys from 16 g on
            const uint4 x = make_uint4(to[v_word(d, 4 * g)], to[v_word(d, 4 * g + 1)],
                                       to[v_word(d, 4 * g + 2)], to[v_word(d, 4 * g + 3)]);
            uint4 *const at = p.v + dst_row * 8 + e;
            const uint32_t got = (uint32_t)(have >> (16 * g)) & 0xffffu;
            if (got == 0xffffu) {
                *at = x;
            } else if (got) {
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int l = 0; l < 16; ++l)
                    if (got >> l & 1)
                        reinterpret_cast<uint8_t *>(at)[perm16(l)] =
                            (uint8_t)(w[perm16(l) / 4] >> (8 * (perm16(l) % 4)));
            }
        }
    }
}

}  // namespace

cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream)
{
    const int64_t ctas = (int64_t)p.R * p.Hkv * ((p.budget + kPage - 1) / kPage);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.fp8 ? compact_kernel<true> : compact_kernel<false>, p);
}

}  // namespace hsa
