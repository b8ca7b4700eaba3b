// kv_select.cu -- the positions of a cache that stay, by accumulated weight (sm_103a).
//
// What it computes: of a row's n weights the first `sinks` positions, the last `recent`, and of
// the rest the left = budget - sinks - recent of the largest score, ties to the lowest position;
// ascending.  A score is the largest weight among a position and its `reach` neighbours.
//
// A score becomes a 32-bit integer of the same order (sign flipped, negatives inverted), its key.
// The left-th largest key is found without a sort, and with no order of atomics that shows: counts
// and prefix sums are exact.
//
// A cluster of 1 to 6 CTAs takes a row, each a contiguous part; a lane takes 16 positions at a time
// (4 of short rows), so that neighbours' weights are read and prefix counts scanned once for all of
// them.
//
// Long rows: two keys of a sample of 2048 positions, five standard deviations of the rank to each
// side, hold the key sought between them.  One pass marks the positions above both and lists those
// between (a few percent); their numbers say whether the rank lies there.  Then the key is found
// digit by digit (8 bits of its distance from the lower bound): a histogram of the digit among the
// listed keys that agree so far, summed from the top until it holds the rank.
//
// Other rows, and those whose sample missed (or whose list did not fit: many ties): the same over
// all positions, digits of 9, 7, 8 and 8 bits.  A thread keeps the high halves of its own keys in
// shared memory, so the passes over them need no barrier, and half as much of it as whole keys
// would: few keys share their high half with the value sought, and only those are made again from
// the weights.  Of those for which there is no room, two bits a key are kept from the third digit
// on.  The first digit, sign and exponent, is every key's, and weights share a few exponents: lanes
// of a warp that add to one counter do so one after another.  So each lane has counters of its own,
// 16 bits wide, in a bank that it shares with one other lane.  The later digits are few keys' and
// differ.
//
// Each CTA writes its counters into the shared memory of all of the cluster (reading the others'
// instead is two round trips and a second barrier a digit, 3 to 6 us).
//
// Then every key above that value stays, and the first `need` keys equal to it, each key's place
// being the number that stay before it (warp scans over contiguous ranges).
//
// What bounds it (the kernel from a cold L2; calls one after the other: 45, 31 and 9 to 10): 16 rows
// of 262144 to 1000000 positions take 48 us (digits over all of them: 75) for 6.4 of HBM: launch and
// sample 14, the pass over the longest row's sixth 17 (instructions: 64 registers a thread, nothing
// loaded ahead), digits 9, places 7.  128 rows of 8192 to 65536 with a reach of 3: 33 (2.8).  8 rows
// of up to 2048: 7, latency.
#include <cooperative_groups.h>

#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 32;
constexpr int kFirstBins = 512;              // of sign and exponent
constexpr int kMaxReach = 7;
constexpr int kMaxCtas = 6;                  // of a row
constexpr int kSampleFrom = 16384;           // positions of a row (4096 to 30000: no difference)
constexpr int kSample = 2048;

struct alignas(16) SelectSmem {              // the held halves follow
    uint32_t lanes[kFirstBins * 16];         // lane l: half l / 16 of word l % 16 of a bin's 16
    uint32_t own[kFirstBins];                // this CTA's counters of a digit
    uint32_t all[2][kMaxCtas][kFirstBins];   // every CTA's, of this digit and the one before
    uint32_t scan[kMaxWarps];
    uint32_t warp_gt[kMaxWarps], warp_eq[kMaxWarps];
    uint32_t cta_gt[kMaxCtas], cta_eq[kMaxCtas];
    uint32_t digit, need;
    int32_t done;
    uint32_t bound[2], rest[2];              // of the sample: digits, and the ranks inside them
    uint32_t listed, above;
};
static_assert(sizeof(SelectSmem) % 16 == 0, "the halves behind it");

// An integer of the value's order; NaN as -infinity, -0 as 0.  Never 0, which marks a position
// that does not compete.
__device__ __forceinline__ uint32_t order_key(float x)
{
    x = x != x ? -INFINITY : x + 0.f;
    const uint32_t u = __float_as_uint(x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Scores of the kKeys positions from p (a multiple of them) of a row of n weights (16-byte aligned,
// readable up to a multiple of 4).
template <int kKeys>
__device__ __forceinline__ void load_scores(float (&v)[kKeys], const float *row, int p, int n, int reach)
{
    float x[kKeys + 16];  // positions p - 8 .. p + 23
#pragma unroll
    for (int c = 0; c < kKeys / 4 + 4; ++c) {
        const int at = p - 8 + 4 * c;
        const bool inner = c >= 2 && c < kKeys / 4 + 2, near = c >= 1 && c < kKeys / 4 + 3;
        float4 y = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if ((inner || (near ? reach > 0 : reach > 4)) && at >= 0 && at < n)
            y = __ldg(reinterpret_cast<const float4 *>(row + at));
        x[4 * c] = y.x, x[4 * c + 1] = y.y, x[4 * c + 2] = y.z, x[4 * c + 3] = y.w;
    }
    if (p + kKeys + 8 > n) {  // behind the row's end
#pragma unroll
        for (int e = 8; e < kKeys + 16; ++e)
            x[e] = p - 8 + e < n ? x[e] : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < kKeys; ++e)
        v[e] = x[8 + e];
#pragma unroll
    for (int d = 1; d <= kMaxReach; ++d)
        if (d <= reach)
#pragma unroll
            for (int e = 0; e < kKeys; ++e)
                v[e] = fmax3(v[e], x[8 + e - d], x[8 + e + d]);  // a NaN gives way to a number
}

// Their keys; those outside lo .. hi - 1 do not compete.
template <int kKeys>
__device__ __forceinline__ void load_keys(uint32_t (&k)[kKeys], const float *row, int p, int n, int lo, int hi,
                                          int reach)
{
    float v[kKeys];
    load_scores<kKeys>(v, row, p, n, reach);
#pragma unroll
    for (int e = 0; e < kKeys; ++e)
        k[e] = order_key(v[e]);
    if (p < lo || p + kKeys > hi) {
#pragma unroll
        for (int e = 0; e < kKeys; ++e)
            if (p + e < lo || p + e >= hi)
                k[e] = 0;
    }
}

// The key of a position that competes.
__device__ __forceinline__ uint32_t one_key(const float *row, int p, int n, int reach)
{
    float v = __ldg(row + p);
    for (int d = 1; d <= reach; ++d)
        v = fmax3(v, p >= d ? __ldg(row + p - d) : -INFINITY, p + d < n ? __ldg(row + p + d) : -INFINITY);
    return order_key(v);
}

// The value of a key.
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k >> 31 ? k ^ 0x80000000u : ~k);
}

template <int kThreads, int kKeys>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) select_kernel(const SelectParams p)
{
    constexpr int kWarps = kThreads / 32;
    constexpr int kChunk = 32 * kKeys;  // positions a warp takes at a time
    constexpr uint32_t kAll = (1u << kKeys) - 1;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SelectSmem &sh = *reinterpret_cast<SelectSmem *>(smem_raw);
    uint32_t *const held = reinterpret_cast<uint32_t *>(smem_raw + sizeof(SelectSmem));
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row_id = blockIdx.x / C, r = row_id / p.heads, h = row_id % p.heads;
    grid_dependency_wait();

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
    if (C > 1)  // every CTA of the cluster runs, before another writes into its shared memory
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // ---- this warp's positions: chunks k_begin .. k_end - 1 ----------------------------------
    const float *const row = p.w + ((int64_t)seq * p.heads + h) * p.w_stride;
    const int chunks = (n + kChunk - 1) / kChunk;
    const int cta_chunks = (chunks + C - 1) / C, warp_chunks = (cta_chunks + kWarps - 1) / kWarps;
    const int k0 = min(chunks, rank * cta_chunks), k1 = min(chunks, k0 + cta_chunks);
    const int k_begin = min(k1, k0 + warp * warp_chunks), k_end = min(k1, k_begin + warp_chunks);
    if (kKeys == 16 && k_begin < k_end && elect_one()) {  // into L2 (43 -> 41 us for 32 x 4 rows of 8192 to 65536)
        const int at = k_begin * kChunk, end = min(k_end * kChunk, (n + 3) & ~3);
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(row + at), "r"((end - at) * 4));
    }
    const int held_chunks = p.held / kChunk;
    // word e of this lane's high halves of chunk c: keys 2 e, 2 e + 1
    auto slot = [&](int c) { return held + (c - k0) * (kChunk / 2) + lane; };
    // of the chunks behind those, a word a lane from the third digit on (in the first's counters):
    // its marks, as below, by high half
    constexpr int kTail = kFirstBins * 16 / 32;
    auto in_tail = [&](int c) { return c - k0 >= held_chunks && c - k0 < held_chunks + kTail; };
    auto tail = [&](int c) { return sh.lanes + (c - k0 - held_chunks) * 32 + lane; };
    auto position = [&](int c) { return c * kChunk + lane * kKeys; };
    auto fresh = [&](int c, uint32_t(&k)[kKeys]) { load_keys<kKeys>(k, row, position(c), n, lo, hi, p.reach); };
    // bit e: the high half of key e, as far as `bits` says, is `value`
    auto match = [&](int c, uint32_t bits, uint32_t value) {
        const uint32_t *const x = slot(c);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < kKeys / 2; ++e) {
            const uint32_t y = x[32 * e] ^ (value | value << 16);
            m |= (y & bits) == 0 ? 1u << (2 * e) : 0u;
            m |= (y & bits << 16) == 0 ? 2u << (2 * e) : 0u;
        }
        return m;
    };

    // exclusive sum over the threads before (the first 512 of them at most hold anything); a barrier
    auto sum_before = [&](uint32_t mine) {
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
        const uint32_t w = lane < warp ? sh.scan[lane] : 0u;
        return incl - mine + __reduce_add_sync(0xffffffffu, w);
    };
    bool waited = C == 1;
    auto may_push = [&] {
        if (!waited)
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        waited = true;
    };

    // ---- long rows: between two keys of a sample ----------------------------------------------
    uint32_t prefix = 0, need = (uint32_t)left, low = 0;
    bool listed = false;
    int shift = 32, list_size = 0;
    uint32_t *const mark = held;  // a word a lane and chunk
    uint2 *const list = reinterpret_cast<uint2 *>(held + cta_chunks * 32);
    const int room = p.held / 4 - cta_chunks * 16;
    if (kKeys == 16 && n >= kSampleFrom && room >= 256) {
        constexpr int kRounds = kSample / 2 / kThreads;
        uint32_t k2[kRounds][2];
        const int spans = (n + kKeys - 1) / kKeys;
        int there = 0;
#pragma unroll
        for (int e = 0; e < kRounds; ++e) {
            uint32_t k[kKeys];
            const int at = (int)((int64_t)(e * kThreads + tid) * spans / (kRounds * kThreads));
            load_keys<kKeys>(k, row, at * kKeys, n, lo, hi, p.reach);
            k2[e][0] = k[0];
            k2[e][1] = k[kKeys / 2];
            there += (k2[e][0] != 0) + (k2[e][1] != 0);
        }
        if (tid < kFirstBins)
            sh.own[tid] = 0;
        if (tid == 0)
            sh.listed = sh.above = 0;
        there = (int)__reduce_add_sync(0xffffffffu, (uint32_t)there);
        if (lane == 0)
            sh.warp_gt[warp] = (uint32_t)there;
        __syncthreads();
        there = (int)__reduce_add_sync(0xffffffffu, lane < kWarps ? sh.warp_gt[lane] : 0u);
#pragma unroll
        for (int e = 0; e < 2 * kRounds; ++e)
            if (k2[e >> 1][e & 1] != 0)
                atomicAdd(&sh.own[k2[e >> 1][e & 1] >> 23], 1u);
        // five standard deviations of the rank on each side
        const float share = (float)left / (float)(hi - lo), mean = share * (float)there;
        const float dev = 5.f * sqrtf(mean * (1.f - share)) + 3.f;
        const int ra = (int)(mean - dev), rb = (int)(mean + dev) + 1;
        if (tid < 2) {  // where there is no such rank: no bound
            sh.bound[tid] = tid == 0 ? 0xffffu : 0u;
            sh.rest[tid] = 0;
        }
        __syncthreads();
        uint32_t mine = tid < kFirstBins ? sh.own[kFirstBins - 1 - tid] : 0u;
        uint32_t before = sum_before(mine);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int rank_e = e == 0 ? ra : rb;
            if (rank_e >= 1 && rank_e <= there && (int)before < rank_e && (int)(before + mine) >= rank_e) {
                sh.bound[e] = (uint32_t)(kFirstBins - 1 - tid);
                sh.rest[e] = (uint32_t)rank_e - before;
            }
        }
        __syncthreads();
        const uint32_t da = sh.bound[0], db = sh.bound[1], na = sh.rest[0], nb = sh.rest[1];
        if (tid < 256)
            sh.own[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2 * kRounds; ++e) {
            const uint32_t k = k2[e >> 1][e & 1];
            if (na != 0 && k >> 23 == da)
                atomicAdd(&sh.own[k >> 16 & 127], 1u);
            if (nb != 0 && k >> 23 == db)
                atomicAdd(&sh.own[128 + (k >> 16 & 127)], 1u);
        }
        __syncthreads();
        mine = tid < 256 ? sh.own[(tid & 128) + 127 - (tid & 127)] : 0u;
        before = sum_before(mine);
        if (tid == 128)
            sh.digit = before;
        __syncthreads();
        if (tid < 256) {
            const int e = tid >> 7;
            const uint32_t b = before - (e ? sh.digit : 0u), want = e ? nb : na;
            if (want != 0 && b < want && b + mine >= want)
                sh.bound[e] = (e ? db : da) << 7 | (uint32_t)(127 - (tid & 127));
        }
        __syncthreads();
        const uint32_t high = sh.bound[0] << 16 | 0xffffu;
        low = max(sh.bound[1] << 16, 1u);

        // the positions above, and a list of those between
        uint32_t gt = 0;
        // (compared as values: bounds that are no numbers, where there is none, hold nothing, and the
        // numbers below then tell)
        const float above_v = key_value(high), level_v = key_value(low);
        for (int c = k_begin; c < k_end; ++c) {
            float v[kKeys];
            uint32_t above = 0, level = 0;
            const int at = position(c);
            load_scores<kKeys>(v, row, at, n, p.reach);
#pragma unroll
            for (int e = 0; e < kKeys; ++e) {
                above |= v[e] > above_v ? 1u << e : 0u;
                level |= v[e] >= level_v ? 1u << e : 0u;
            }
            if (at < lo || at + kKeys > hi) {
                const uint32_t in = (hi - at >= kKeys ? kAll : hi > at ? (1u << (hi - at)) - 1 : 0u) &
                                    (lo <= at ? kAll : lo - at < kKeys ? kAll << (lo - at) : 0u);
                above &= in;
                level &= in;
            }
            level &= ~above;
            mark[(c - k0) * 32 + lane] = above;
            gt += __popc(above);
            if (!__any_sync(0xffffffffu, level != 0))
                continue;
            const uint32_t count = __popc(level);
            uint32_t incl = count;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += u;
            }
            uint32_t to = 0;
            if (lane == 31)
                to = atomicAdd(&sh.listed, incl);
            to = __shfl_sync(0xffffffffu, to, 31) + incl - count;
            for (uint32_t m = level; m; m &= m - 1, ++to)
                if (to < (uint32_t)room)
                    list[to].y = (uint32_t)((c - k0) * kChunk + lane * kKeys + __ffs(m) - 1);
        }
        gt = __reduce_add_sync(0xffffffffu, gt);
        if (lane == 0 && gt != 0)
            atomicAdd(&sh.above, gt);
        __syncthreads();
        list_size = min((int)sh.listed, room);
        for (int i = tid; i < list_size; i += kThreads)
            list[i].x = one_key(row, k0 * kChunk + (int)list[i].y, n, p.reach);
        uint32_t total_gt = sh.above, total = sh.listed;
        bool fits = total <= (uint32_t)room;
        if (C > 1) {
            may_push();
            if (tid < C) {
                *cluster.map_shared_rank(&sh.cta_gt[rank], tid) = total_gt;
                *cluster.map_shared_rank(&sh.cta_eq[rank], tid) = fits ? total : 1u << 30;
            }
            cluster.sync();
            total_gt = total = 0;
            for (int c = 0; c < C; ++c) {
                total_gt += sh.cta_gt[c];
                total += min(sh.cta_eq[c], 1u << 28);
                fits &= sh.cta_eq[c] != 1u << 30;
            }
        }
        listed = fits && total_gt < (uint32_t)left && total_gt + total >= (uint32_t)left;
        if (!listed)
            low = 0;  // every key, as if there had been no sample
        if (listed) {
            need = (uint32_t)left - total_gt;
            shift = max((39 - __clz(high - low)) / 8, 1) * 8;  // digits of eight bits of key - low
        }
        __syncthreads();
    }

    // ---- the left-th largest key, digit by digit --------------------------------------------
    bool tailed = false;
    bool exact = false;  // need ends inside the digit's keys (else all of them stay)
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int bits = listed ? 8 : pass == 0 ? 9 : pass == 1 ? 7 : 8, bins = 1 << bits;
        const int above = shift;  // bits above the digit agree with prefix
        shift -= bits;
        if (listed) {
            if (tid < bins)
                sh.own[tid] = 0;
            __syncthreads();
            for (int i = tid; i < list_size; i += kThreads) {
                const uint32_t k = list[i].x - low;
                if (pass == 0 || k >> above == prefix)
                    atomicAdd(&sh.own[k >> shift & 255], 1u);
            }
        } else if (pass == 0) {
            for (int b = tid; b < kFirstBins * 4; b += kThreads)
                reinterpret_cast<uint4 *>(sh.lanes)[b] = make_uint4(0, 0, 0, 0);
            __syncthreads();
            const uint32_t one = lane < 16 ? 1u : 0x10000u;
            for (int c = k_begin; c < k_end; ++c) {
                uint32_t k[kKeys];
                fresh(c, k);
                if (c - k0 < held_chunks) {
                    uint32_t *const x = slot(c);
#pragma unroll
                    for (int e = 0; e < kKeys / 2; ++e)
                        x[32 * e] = __byte_perm(k[2 * e], k[2 * e + 1], 0x7632);
                }
#pragma unroll
                for (int e = 0; e < kKeys; ++e)
                    if (k[e] != 0)
                        atomicAdd(&sh.lanes[(k[e] >> 23) * 16 + (lane & 15)], one);
            }
            __syncthreads();
            for (int b = tid; b < kFirstBins; b += kThreads) {
                uint32_t sum = 0;
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const uint32_t x = sh.lanes[b * 16 + ((j + b) & 15)];
                    sum += (x & 0xffffu) + (x >> 16);
                }
                sh.own[b] = sum;
            }
        } else {
            for (int b = tid; b < bins; b += kThreads)
                sh.own[b] = 0;
            __syncthreads();
            // (few keys agree with the digits so far: bits are cheaper than a branch for each)
            const uint32_t known = above >= 16 ? 0xffffu << (above - 16) & 0xffffu : 0xffffu;
            const uint32_t half = above >= 16 ? prefix << (above - 16) : prefix >> (16 - above);
            for (int c = k_begin; c < k_end; ++c) {
                const bool there = c - k0 < held_chunks;
                uint32_t m = there ? match(c, known, half) : pass == 3 && in_tail(c) ? *tail(c) >> 16 : kAll;
                if (pass == 1 && there) {
                    for (; m; m &= m - 1) {
                        const int e = __ffs(m) - 1;
                        const uint32_t k = slot(c)[32 * (e >> 1)] >> (16 * (e & 1)) & 0xffffu;
                        if (k != 0)
                            atomicAdd(&sh.own[k & (bins - 1)], 1u);
                    }
                } else if (m) {
                    uint32_t k[kKeys];
                    fresh(c, k);
                    if (pass == 2 && in_tail(c)) {
                        uint32_t x = 0;
#pragma unroll
                        for (int e = 0; e < kKeys; ++e) {
                            x |= k[e] >> 16 > prefix ? 1u << e : 0u;
                            x |= k[e] >> 16 == prefix ? 0x10000u << e : 0u;
                        }
                        *tail(c) = x;
                    }
#pragma unroll
                    for (int e = 0; e < kKeys; ++e)
                        if (k[e] != 0 && (k[e] >> above) == prefix)
                            atomicAdd(&sh.own[(k[e] >> shift) & (bins - 1)], 1u);
                }
            }
        }
        tailed = !listed && pass >= 2;
        __syncthreads();
        const uint32_t(*const all)[kFirstBins] = sh.all[pass & 1];
        if (C > 1) {
            may_push();
            for (int i = tid; i < C * (bins / 4); i += kThreads) {
                const int to = i / (bins / 4), at = i % (bins / 4);
                reinterpret_cast<uint4 *>(cluster.map_shared_rank(sh.all[pass & 1][rank], to))[at] =
                    reinterpret_cast<const uint4 *>(sh.own)[at];
            }
            cluster.sync();  // (and all have read what was written two digits ago)
        }
        // the digit that holds the rank: a counter a thread, the top one in thread 0
        static_assert(kThreads >= kFirstBins, "a counter a thread");
        uint32_t mine = 0;
        if (tid < bins) {
            if (C == 1) {
                mine = sh.own[bins - 1 - tid];
            } else {
#pragma unroll
                for (int c = 0; c < kMaxCtas; ++c)
                    mine += c < C ? all[c][bins - 1 - tid] : 0u;
            }
        }
        const uint32_t before = sum_before(mine);
        if (tid < bins) {
            if (before < need && before + mine >= need) {  // one thread
                sh.digit = (uint32_t)(bins - 1 - tid);
                sh.need = need - before;
                sh.done = need - before == mine;
            }
        }
        __syncthreads();
        prefix = (prefix << bits) | sh.digit;
        need = sh.need;
        if (sh.done)  // (the next digit's counts come behind a barrier)
            break;
        exact = shift == 0;
        if (exact)
            break;
    }
    // keys above `edge` stay, and of those equal to it the first `need` (none: the last digit's
    // keys all stay, and edge is the value below them)
    const uint32_t edge = exact ? low + prefix : max(low + (prefix << shift), 1u) - 1u;
    if (!exact)
        need = 0;
    if (listed) {
        for (int i = tid; i < list_size; i += kThreads) {
            const uint2 x = list[i];
            if (x.x > edge || (x.x == edge && need != 0))
                atomicOr(&mark[x.y >> 4], (x.x > edge ? 1u : 0x10000u) << (x.y & 15));
        }
        __syncthreads();
    }

    // ---- which stay: bit e of a word key e above the edge, bit 16 + e equal to it -----------
    const uint32_t edge16 = edge >> 16;
    auto marks = [&](int c) {
        if (listed)
            return mark[(c - k0) * 32 + lane];
        uint32_t above = 0, level = kAll;
        if (c - k0 < held_chunks) {
            const uint32_t *const x = slot(c);
            level = 0;
#pragma unroll
            for (int e = 0; e < kKeys; ++e) {
                const uint32_t y = e & 1 ? x[32 * (e >> 1)] >> 16 : x[32 * (e >> 1)] & 0xffffu;
                above |= y > edge16 ? 1u << e : 0u;
                level |= y == edge16 ? 1u << e : 0u;
            }
        } else if (tailed && in_tail(c)) {
            const uint32_t x = *tail(c);
            above = x & 0xffffu;
            level = x >> 16;
        }
        if (level) {  // a high half that does not tell
            uint32_t k[kKeys];
            fresh(c, k);
            above = level = 0;
#pragma unroll
            for (int e = 0; e < kKeys; ++e) {
                above |= k[e] > edge ? 1u << e : 0u;
                level |= k[e] == edge && k[e] != 0 ? 0x10000u << e : 0u;
            }
        }
        return above | level;
    };
    uint32_t gt = 0, eq = 0;
    for (int c = k_begin; c < k_end; ++c) {
        const uint32_t x = marks(c);
        if (listed)
            ;
        else if (c - k0 < held_chunks)
            *slot(c) = x;  // the halves are not needed any more
        else if (in_tail(c))
            *tail(c) = x;
        gt += __popc(x & 0xffffu);
        eq += __popc(x >> 16);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        sh.warp_gt[warp] = gt;
        sh.warp_eq[warp] = eq;
    }
    __syncthreads();
    if (C > 1) {
        if (tid < C) {
            uint32_t g = 0, e = 0;
            for (int w = 0; w < kWarps; ++w) {
                g += sh.warp_gt[w];
                e += sh.warp_eq[w];
            }
            *cluster.map_shared_rank(&sh.cta_gt[rank], tid) = g;
            *cluster.map_shared_rank(&sh.cta_eq[rank], tid) = e;
        }
        cluster.sync();
    }
    uint32_t g0 = 0, e0 = 0;
    for (int c = 0; c < rank; ++c) {
        g0 += sh.cta_gt[c];
        e0 += sh.cta_eq[c];
    }
    for (int w = 0; w < warp; ++w) {
        g0 += sh.warp_gt[w];
        e0 += sh.warp_eq[w];
    }

    // ---- the positions, each at the number that stay before it ------------------------------
    int32_t *const to = keep + p.sinks;
    for (int c = k_begin; c < k_end; ++c) {
        const uint32_t x = listed ? marks(c) : c - k0 < held_chunks ? *slot(c) : in_tail(c) ? *tail(c) : marks(c);
        const uint32_t mine = __popc(x & 0xffffu) | __popc(x >> 16) << 16;
        uint32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += y;
        }
        uint32_t g = g0 + ((incl - mine) & 0xffffu), e2 = e0 + ((incl - mine) >> 16);
        if (need == 0) {
            for (uint32_t m = x & 0xffffu; m; m &= m - 1)
                to[g++] = position(c) + __ffs(m) - 1;
        } else {
            for (uint32_t m = (x | x >> 16) & 0xffffu; m; m &= m - 1) {
                const int e = __ffs(m) - 1;
                const bool above = x >> e & 1;
                if (above || e2 < need)
                    to[g + min(e2, need)] = position(c) + e;
                g += above;
                e2 += !above;
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
    // CTAs a row: as many as fill the SMs, with one CTA of 1024 threads each (64 registers a thread:
    // they take all of an SM's) or, for more rows than SMs, two of 512 (128 rows: 33 us with a whole
    // SM each, 40 with two halves of one that exchange); 2048 positions a CTA at least (8192: the
    // same), and 2^20 at most, for a lane's 16-bit counters (api.cu holds w_stride to 2^22).  At most
    // six: 23 clusters of six such CTAs find room at once, but 15 of seven or of eight, and the
    // sixteenth of 16 rows began 34 us late.
    const bool small = p.w_stride <= 8192;
    const bool wide = rows <= sms && !small;
    int64_t C = (wide ? 1 : 2) * sms / rows;
    C = C < kMaxCtas ? C : kMaxCtas;
    C = C < p.w_stride / 2048 ? C : p.w_stride / 2048;
    C = C > (p.w_stride >> 20) + 1 ? C : (p.w_stride >> 20) + 1;
    const int chunk = 32 * (small ? 4 : 16);
    const int64_t chunks = ((int64_t)p.w_stride + chunk - 1) / chunk, per = (chunks + C - 1) / C * chunk;
    // of an SM's 227 KB, for one CTA or for two
    const int64_t most = ((wide ? 224 : 112) * 1024 - (int64_t)sizeof(SelectSmem)) / (2 * chunk) * chunk;
    p.held = (int32_t)(per < most ? per : most);
    const size_t smem = sizeof(SelectSmem) + (size_t)p.held * 2;
    static SmemOptIn opt[3];
    const auto kern = small ? select_kernel<512, 4> : wide ? select_kernel<1024, 16> : select_kernel<512, 16>;
    const cudaError_t e = opt[small ? 0 : wide ? 1 : 2].set(kern, 224 * 1024);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(rows * C));
    cfg.blockDim = dim3(wide ? 1024 : 512);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace hsa
