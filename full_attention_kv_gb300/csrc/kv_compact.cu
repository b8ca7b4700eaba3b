// kv_compact.cu -- the rows of a full layer that stay, moved into pages of their own (sm_103a).
//
// What it does: for request r, KV head h and i < new_len[r], the K and V rows (and the weight) at
// position keep[r][h][i] of the sequence go to position i of the pages dst_tables[r].  Stored
// values move as they are: bf16 rows, or an FP8 layer's codes and scales (fp8_kv.cuh).
//
// One CTA a destination page of a head.  Its 64 source rows are found first (keep, then the block
// table), then every 16-byte chunk is one thread's: 256 contiguous bytes a bf16 row, 128 an FP8 K
// row.  An FP8 layer's V is stored transposed (64 keys of a dimension side by side), so a single
// key is 128 bytes in as many sectors; the source pages are taken whole instead (positions ascend,
// so a page's keys are neighbours in the list), 8 KB bulk copies into shared memory, kPages of them
// at a time.  A lane then puts together the same four keys of eight dimensions: two rows of 64 bytes
// a warp, which meet 32 banks whatever the keys, and leave as 128 contiguous bytes.
//
// What bounds it: HBM.  16 requests of 4096 rows x 4 heads, bf16: 45 us, 0.89 of a copy's rate.  FP8 (8
// requests of 2000 rows out of 3000 to 9000): 19 us from a cold L2 (12 where it holds the pages), 38
// MB read for 17 kept, and the pages' latency.
#include "fp8_kv.cuh"
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kThreads = 256;
constexpr int kPage = 64;

constexpr int kPages = 6;               // source pages of V held at a time
constexpr int kPageBytes = kPage * 128; // FP8 codes

// Byte of key `row` of a page in a V row.
__device__ __forceinline__ int v_byte(int row) { return 16 * (row >> 4) + perm16(row & 15); }

struct VPages {
    alignas(128) uint8_t stage[kPages][kPageBytes];
    alignas(8) uint64_t full;
    int64_t page[kPage];  // pages in the order of the list
    int32_t slot[kPage];  // each key's among them
    int32_t n;
};

template <bool FP8>
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactParams p)
{
    __shared__ int64_t src[kPage];  // a head's row in the pool, or -1
    __shared__ uint32_t ok[2];      // bit i: row i is to be copied
    extern __shared__ __align__(128) uint8_t smem_raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pages = (p.budget + kPage - 1) / kPage;
    const int page = blockIdx.x % pages;
    const int64_t rh = blockIdx.x / pages;
    const int h = (int)(rh % p.Hkv), r = (int)(rh / p.Hkv);
    grid_dependency_wait();

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
        // ---- V: the source pages, one for each run of the list ------------------------------
        VPages &sh = *reinterpret_cast<VPages *>(smem_raw);
        if (tid == 0) {
            mbar_init(&sh.full, 1);
            fence_barrier_init();
        }
        if (tid < kPage) {
            const int64_t pg = src[tid] >= 0 ? src[tid] / kPage : -1;
            int64_t last = -1;  // the page of the nearest row before that is copied
            const uint64_t have = (uint64_t)ok[1] << 32 | ok[0], below = have & ((1ull << tid) - 1);
            if (below)
                last = src[63 - __clzll((long long)below)] / kPage;
            const bool starts = pg >= 0 && pg != last;
            const uint32_t bits = __ballot_sync(0xffffffffu, starts);
            if (lane == 0)
                sh.slot[warp] = __popc(bits);
            named_bar_sync(1, kPage);
            const int before = warp == 1 ? sh.slot[0] : 0, all = sh.slot[0] + sh.slot[1];
            named_bar_sync(1, kPage);
            const int at = before + __popc(bits & (2u << lane) - 1u) - 1;
            sh.slot[tid] = pg >= 0 ? at : -1;
            if (starts)
                sh.page[at] = pg;
            if (tid == 0)
                sh.n = all;
        }
        __syncthreads();
        auto fetch = [&](int s0) {
            if (tid == 0 && s0 < sh.n && !kWithholdLoads) {
                const int n = min(kPages, sh.n - s0);
                mbar_arrive_expect_tx(&sh.full, n * kPageBytes);
                for (int e = 0; e < n; ++e)
                    bulk_load(sh.stage[e], p.v + sh.page[s0 + e] * 512, kPageBytes, &sh.full, policy_evict_first());
            }
        };
        fetch(0);
        // ---- K rows and the scales, meanwhile -----------------------------------------------
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
        // this lane's word of a V row: four keys, each a slot and a byte there
        const int word = lane & 15;
        int slot[4], off[4];
        bool whole = true, some = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // byte e of the word is this key (perm16 undone)
            const int key = 16 * (word >> 2) + 2 * (word & 3) + (e & 1) + 8 * (e >> 1);
            slot[e] = sh.slot[key];
            off[e] = slot[e] >= 0 ? v_byte((int)(src[key] % kPage)) : 0;
            whole &= slot[e] >= 0;
            some |= slot[e] >= 0;
        }
        uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        bool done = true;
        for (int s0 = 0, phase = 0; s0 < sh.n; s0 += kPages, phase ^= 1) {
            if (!mbar_wait(&sh.full, phase)) {
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
                done = false;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int st = slot[e] - s0;
                if (slot[e] >= 0 && st >= 0 && st < kPages) {
                    const uint8_t *const from = &sh.stage[st][(2 * warp + (lane >> 4)) * 64 + off[e]];
#pragma unroll
                    for (int j = 0; j < 8; ++j)  // dimensions 16 apart
                        x[j] |= (uint32_t)from[j * 1024] << (8 * e);
                }
            }
            done = __syncthreads_and(done);  // the stages are free again
            if (!done) {
                mbar_wait(&sh.full, phase);  // no copy may still be in flight when the CTA exits
                break;
            }
            fetch(s0 + kPages);
        }
        uint32_t *const to = reinterpret_cast<uint32_t *>(p.v + dst_row * 8) + (2 * warp + (lane >> 4)) * 16 + word;
        if (done && some) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (whole) {
                    to[j * 256] = x[j];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (slot[e] >= 0)
                            reinterpret_cast<uint8_t *>(to + j * 256)[e] = (uint8_t)(x[j] >> (8 * e));
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_compact(const CompactParams &p, cudaStream_t stream)
{
    const int64_t ctas = (int64_t)p.R * p.Hkv * ((p.budget + kPage - 1) / kPage);
    const size_t smem = p.fp8 ? sizeof(VPages) : 0;
    static SmemOptIn opt;
    if (p.fp8) {
        const cudaError_t e = opt.set(compact_kernel<true>, smem);
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, p.fp8 ? compact_kernel<true> : compact_kernel<false>, p);
}

}  // namespace hsa
