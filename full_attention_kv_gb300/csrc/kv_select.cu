// kv_select.cu -- the positions of a cache that stay, by accumulated weight (sm_103a).
//
// What it computes: of a row's n weights the first `sinks` positions, the last `recent`, and of
// the rest the left = budget - sinks - recent of the largest score, ties to the lowest position;
// ascending.  A score is the largest weight among a position and its `reach` neighbours.
//
// A score becomes a 32-bit integer of the same order (sign flipped, negatives inverted), and the
// left-th largest is found digit by digit (11, 11 and 10 bits): a histogram of the digit among
// the keys that agree so far, summed from the top until it holds the rank.  No sort, and no
// order of atomics that shows: the histogram's sums and the prefix counts are exact.  Then every
// key above that value stays, and the first `need` keys equal to it, each key's place being the
// number that stay before it (warp scans over contiguous ranges).
//
// A cluster of 1 to 8 CTAs takes a row, each a contiguous part, read from memory once: a thread
// keeps its own keys in shared memory (as far as they fit; the others are read again, out of
// L2), so the passes over them need no barrier.  Histograms are summed over the cluster through
// distributed shared memory.
#include <cooperative_groups.h>

#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxReach = 7;

struct alignas(16) SelectSmem {  // the held keys follow
    uint32_t hist[kBins];
    uint32_t scan[kWarps];
    uint32_t warp_gt[kWarps], warp_eq[kWarps];
    uint32_t cta_gt, cta_eq;
    uint32_t digit, need;
    int32_t done;
};
static_assert(sizeof(SelectSmem) % 16 == 0, "the keys behind it are read 16 bytes at a time");

// An integer of the value's order; NaN as -infinity, -0 as 0.  Never 0, which marks a position
// that does not compete.
__device__ __forceinline__ uint32_t order_key(float x)
{
    x = x != x ? -INFINITY : x + 0.f;
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Keys of positions 4 quad .. 4 quad + 3 of a row of n weights (16-byte aligned, readable up to
// a multiple of 4); those outside lo .. hi - 1 do not compete.
__device__ __forceinline__ uint4 load_keys(const float *row, int quad, int n, int lo, int hi, int reach)
{
    const int p = 4 * quad;
    float v[4];
    if (reach == 0) {
        const float4 x = __ldg(reinterpret_cast<const float4 *>(row) + quad);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        float x[20];  // positions p - 8 .. p + 11
#pragma unroll
        for (int c = 0; c < 5; ++c) {
            const int at = p - 8 + 4 * c;
            float4 y = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (at >= 0 && at < n)
                y = __ldg(reinterpret_cast<const float4 *>(row + at));
            x[4 * c] = y.x;
            x[4 * c + 1] = at + 1 < n ? y.y : -INFINITY;
            x[4 * c + 2] = at + 2 < n ? y.z : -INFINITY;
            x[4 * c + 3] = at + 3 < n ? y.w : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = x[8 + e];
#pragma unroll
        for (int d = 1; d <= kMaxReach; ++d)
            if (d <= reach)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = fmax3(v[e], x[8 + e - d], x[8 + e + d]);  // a NaN gives way to a number
    }
    uint32_t k[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        k[e] = p + e >= lo && p + e < hi ? order_key(v[e]) : 0u;
    return make_uint4(k[0], k[1], k[2], k[3]);
}

__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p)
{
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SelectSmem &sh = *reinterpret_cast<SelectSmem *>(smem_raw);
    uint4 *const held = reinterpret_cast<uint4 *>(smem_raw + sizeof(SelectSmem));
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row_id = blockIdx.x / C, r = row_id / p.heads, h = row_id % p.heads;
    grid_dependency_wait();
    grid_launch_dependents();

    const int seq = __ldg(p.seq_idx + r);
    int n = __ldg(p.kv_len + r);
    int err = 0;
    if (seq < 0 || seq >= p.batch)
        err = HSA_DEVERR_BAD_SEQ;
    else if (n < 0 || n > p.w_stride)
        err = HSA_DEVERR_BAD_LEN;
    if (err) {
        n = 0;
        if (tid == 0 && rank == 0 && h == 0)
            set_err(p.dev_err, err);
    }
    int32_t *const keep = p.keep + (int64_t)row_id * p.budget;
    if (tid == 0 && rank == 0 && h == 0)
        p.new_len[r] = min(n, p.budget);
    if (n <= p.budget) {  // the same for the whole cluster
        for (int i = rank * kThreads + tid; i < p.budget; i += C * kThreads)
            keep[i] = i < n ? i : -1;
        return;
    }
    const int lo = p.sinks, hi = n - p.recent;
    const int left = p.budget - p.sinks - p.recent;
    for (int i = rank * kThreads + tid; i < p.sinks; i += C * kThreads)
        keep[i] = i;
    for (int i = rank * kThreads + tid; i < p.recent; i += C * kThreads)
        keep[p.budget - p.recent + i] = hi + i;
    if (left == 0)
        return;

    // ---- this thread's quads of positions: q_begin + lane, + 32, ... < q_end ----------------
    const float *const row = p.w + ((int64_t)seq * p.heads + h) * p.w_stride;
    const int quads = (n + 3) / 4;
    const int per_cta = (quads + C - 1) / C;
    const int c0 = min(quads, rank * per_cta), c1 = min(quads, c0 + per_cta);
    const int per_warp = ((per_cta + kWarps - 1) / kWarps + 31) & ~31;
    const int q_begin = min(c1, c0 + warp * per_warp), q_end = min(c1, q_begin + per_warp);
    const int held_quads = p.held / 4;
    auto keys = [&](int q) {
        return q - c0 < held_quads ? held[q - c0] : load_keys(row, q, n, lo, hi, p.reach);
    };

    // ---- the left-th largest key, digit by digit --------------------------------------------
    uint32_t prefix = 0, need = (uint32_t)left;
    bool exact = false;  // need ends inside the digit's keys (else all of them stay)
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        const int above = shift;  // bits above the digit agree with prefix
        shift -= bits;
        for (int b = tid; b < kBins; b += kThreads)
            sh.hist[b] = 0;
        __syncthreads();
        for (int q = q_begin + lane; q < q_end; q += 32) {
            uint4 k4;
            if (pass == 0) {
                k4 = load_keys(row, q, n, lo, hi, p.reach);
                if (q - c0 < held_quads)
                    held[q - c0] = k4;
            } else {
                k4 = keys(q);
            }
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (k[e] != 0 && (pass == 0 || (k[e] >> above) == prefix))
                    atomicAdd(&sh.hist[(k[e] >> shift) & ((1u << bits) - 1)], 1u);
        }
        if (C > 1)
            cluster.sync();
        else
            __syncthreads();
        // thread t sums bins 2047 - 4t .. 2044 - 4t over the cluster: the top ones first
        uint32_t cnt[4] = {0, 0, 0, 0};
        const int b0 = kBins - 4 - 4 * tid;
#pragma unroll 1
        for (int c = 0; c < C; ++c) {
            const uint4 x = *reinterpret_cast<const uint4 *>(
                C > 1 ? cluster.map_shared_rank(&sh.hist[b0], c) : &sh.hist[b0]);
            cnt[0] += x.w, cnt[1] += x.z, cnt[2] += x.y, cnt[3] += x.x;
        }
        const uint32_t mine = cnt[0] + cnt[1] + cnt[2] + cnt[3];
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        if (lane == 31)
            sh.scan[warp] = incl;
        __syncthreads();
        uint32_t before = incl - mine;
        for (int w = 0; w < warp; ++w)
            before += sh.scan[w];
        if (before < need && before + mine >= need) {  // one thread
            int e = 0;
            while (before + cnt[e] < need)
                before += cnt[e++];
            sh.digit = (uint32_t)(b0 + 3 - e);
            sh.need = need - before;
            sh.done = need - before == cnt[e];
        }
        if (C > 1)
            cluster.sync();  // every CTA has read the histograms
        else
            __syncthreads();
        prefix = (prefix << bits) | sh.digit;
        need = sh.need;
        if (sh.done)
            break;
        exact = pass == 2;
    }
    // keys above `edge` stay, and of those equal to it the first `need` (none: the last digit's
    // keys all stay, and edge is the value below them)
    const uint32_t edge = exact ? prefix : (prefix << shift) - 1u;
    if (!exact)
        need = 0;

    // ---- how many stay before each warp's range ---------------------------------------------
    uint32_t gt = 0, eq = 0;
    for (int q = q_begin + lane; q < q_end; q += 32) {
        const uint4 k = keys(q);
        gt += (k.x > edge) + (k.y > edge) + (k.z > edge) + (k.w > edge);
        eq += (k.x == edge) + (k.y == edge) + (k.z == edge) + (k.w == edge);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sh.warp_gt[warp] = gt;
        sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, e = 0;
        for (int w = 0; w < kWarps; ++w) {
            g += sh.warp_gt[w];
            e += sh.warp_eq[w];
        }
        sh.cta_gt = g;
        sh.cta_eq = e;
    }
    uint32_t g0 = 0, e0 = 0;
    for (int w = 0; w < warp; ++w) {
        g0 += sh.warp_gt[w];
        e0 += sh.warp_eq[w];
    }
    if (C > 1) {
        cluster.sync();
        for (int c = 0; c < rank; ++c) {
            g0 += *cluster.map_shared_rank(&sh.cta_gt, c);
            e0 += *cluster.map_shared_rank(&sh.cta_eq, c);
        }
        cluster.sync();  // no CTA leaves while its counts are read
    }

    // ---- the positions, each at the number that stay before it ------------------------------
    int32_t *const to = keep + p.sinks;
    for (int q = q_begin; q < q_end; q += 32) {
        uint4 k4 = make_uint4(0, 0, 0, 0);
        if (q + lane < q_end)
            k4 = keys(q + lane);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
        uint32_t c = 0;  // keys above the edge, and equal to it in the high half
#pragma unroll
        for (int e = 0; e < 4; ++e)
            c += (k[e] > edge) + ((uint32_t)(k[e] == edge && k[e] != 0) << 16);
        if (!__any_sync(0xffffffffu, c != 0))
            continue;
        uint32_t incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        uint32_t g = g0 + ((incl - c) & 0xffffu), e2 = e0 + ((incl - c) >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (k[e] > edge) {
                to[g + min(e2, need)] = 4 * (q + lane) + e;
                ++g;
            } else if (k[e] == edge) {
                if (e2 < need)
                    to[g + e2] = 4 * (q + lane) + e;
                ++e2;
            }
        }
        const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
        g0 += all & 0xffffu;
        e0 += all >> 16;
    }
}

}  // namespace

cudaError_t launch_select(SelectParams &p, int sms, cudaStream_t stream)
{
    const int64_t rows = (int64_t)p.R * p.heads;
    // CTAs a row: as many as leave each at least 4096 positions and the grid at most two a SM
    int C = 1;
    while (C < 8 && rows * C <= sms && p.w_stride / C > 4096)
        C *= 2;
    const int per = ((p.w_stride + 3) / 4 + C - 1) / C * 4;
    const int most = (rows * C <= sms ? 200 : 100) * 256;  // KB as keys
    p.held = per < most ? per : most;
    const size_t smem = sizeof(SelectSmem) + (size_t)p.held * 4;
    static SmemOptIn opt;
    const cudaError_t e = opt.set(select_kernel, sizeof(SelectSmem) + 200 * 1024);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_kernel, p);
}

}  // namespace hsa
