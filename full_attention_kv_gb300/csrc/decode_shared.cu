// decode_shared.cu -- decode / MTP-verify attention for groups of sequences that share
// their first pages (sm_103a).
//
// What it computes: what decode.cu computes on a full layer, o = softmax(scale q . K^T) V
// over a sequence's cached keys and its T new ones.  The prefix tree lets sequences share
// pages (a system prompt, a document, samples of one prompt); decode.cu reads those pages
// once for every sequence.  Here a group's shared pages are read once for all of its rows:
// softmax over a union of key sets splits into per-set states (m, l, o) that merge exactly,
//   m = max m_i,  l = sum l_i 2^(m_i - m),  o = sum o_i 2^(m_i - m) / l,
// so the shared pages and each sequence's own pages are separate passes.
//
// Pass 1, shared_kernel (tcgen05): the query rows of a group for one KV head -- members x T
// tokens x G heads -- are packed into 128-row tiles, a pair of tiles (256 rows) a unit, and
// meet the shared keys in 128-key tiles as a dense product: K and V are read once a unit
// instead of once a sequence.  The key tiles of all units are laid end to end and cut into
// equal ranges, one per CTA; each (CTA, unit) segment leaves unnormalised fp32 states.
// Pass 2, own_kernel (mma.sync, 8 to 32 rows a sequence and head): a stream-K walk over the
// pages past the shared ones and the new tokens; each segment leaves its state.
// Pass 3, merge_kernel: a thread for four output dimensions of a row merges the row's
// states and writes bf16; it also appends the new rows.
//
// The passes overlap by programmatic dependent launch: pass 2 reads nothing of pass 1, and
// its CTAs start as pass 1's leave their SMs; pass 3 is resident before pass 2 ends.
#include "decode_tile.cuh"
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

// ------------------------------------------------------------------ groups, both passes

// A group's shared whole pages, or 0 (nothing is shared).
__device__ __forceinline__ int group_pages(const SharedParams &p, int g)
{
    const int len = __ldg(p.shared_len + g);
    return len > 0 ? min(len / kTileKeys, p.d.max_blocks) : 0;
}

// Whether cu_group is 0 = cu[0] <= cu[1] <= ... <= cu[n] = B.  Called by a whole warp.
// Offsets out of order share nothing: every sequence then reads all of its pages itself.
__device__ __forceinline__ bool groups_ok(const SharedParams &p, int lane)
{
    bool ok = true;
    for (int g = lane; g < p.n_groups; g += 32) {
        const int a = __ldg(p.cu_group + g), b = __ldg(p.cu_group + g + 1);
        __ldg(p.shared_len + g);  // wanted next: one latency for all three
        ok = ok && a <= b && (g > 0 || a == 0) && (g + 1 < p.n_groups || b == p.d.B);
    }
    return __all_sync(0xffffffffu, ok) && p.n_groups > 0;
}

// The group of sequence b (offsets in order).
__device__ __forceinline__ int group_of(const SharedParams &p, int b)
{
    int lo = 0, hi = p.n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu_group + mid) <= b)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int clamp_len(int c) { return c < 0 ? 0 : c; }

// ------------------------------------------------------------------ pass 1: shared pages

constexpr int kBM = 128;
constexpr int kBN = 128;
constexpr int kHalfBytes = 128 * 128;       // 128 rows x 64 bf16 (one swizzle column block)
constexpr int kOpBytes = 2 * kHalfBytes;    // 32 KB
constexpr int kSharedThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;             // S_A, S_B at 0 / 128; O_A, O_B at 256 / 384
// A segment's states, by octets of rows: m[8], l[8], then o as [dim / 4][8 rows][4], so
// that the warps that write (a row a lane) and those that merge (eight rows x four
// 16-byte pieces) both move whole 128-byte lines.
constexpr int kOctFloats = 16 + 8 * kD;
constexpr int kSlotFloats = 2 * kBM / 8 * kOctFloats;

struct SharedSmem {
    alignas(1024) uint8_t q[2][kOpBytes];
    alignas(1024) uint8_t k[2][kOpBytes];
    alignas(1024) uint8_t v[2][kOpBytes];
    alignas(8) uint64_t q_full, q_empty;
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
    uint32_t tmem_base;
    int32_t g0, unit0;
    int64_t item0, N;
};

// A CTA's walk over the segments of its item range: every role runs its own copy.
// A unit of at most 128 rows has one query tile; the two softmax warpgroups, S and O
// regions then take its key tiles in turn (split()), so that one tile's products still
// run under the other's softmax, and the segment leaves two states a row.
struct SegWalk {
    int64_t it, i1, item0;  // next item, end, first item of group g
    int g, unit0;           // group, units before it
    int pairs, kt;          // the group's 256-row units a head, 128-key tiles a unit
    int seq0, ntok, pages;
    // the current segment
    int h, pair, n0, n1, unit, rows;
    __device__ __forceinline__ bool split() const { return rows <= kBM; }
};

__device__ __forceinline__ void load_group(const SharedParams &p, SegWalk &w)
{
    w.seq0 = __ldg(p.cu_group + w.g);
    w.ntok = (__ldg(p.cu_group + w.g + 1) - w.seq0) * p.d.T;
    w.pages = group_pages(p, w.g);
    w.kt = (w.pages + 1) >> 1;
    w.pairs = w.kt > 0 ? (w.ntok * p.d.G + 2 * kBM - 1) / (2 * kBM) : 0;
}

__device__ __forceinline__ bool next_seg(const SharedParams &p, SegWalk &w)
{
    if (w.it >= w.i1)
        return false;
    int64_t n = (int64_t)w.pairs * p.d.Hkv * w.kt;
    while (w.it >= w.item0 + n) {
        w.item0 += n;
        w.unit0 += w.pairs * p.d.Hkv;
        ++w.g;
        load_group(p, w);
        n = (int64_t)w.pairs * p.d.Hkv * w.kt;
    }
    const int64_t off = w.it - w.item0;
    const int u = (int)(off / w.kt);
    w.n0 = (int)(off % w.kt);
    w.n1 = (int)min((int64_t)w.kt, w.n0 + (w.i1 - w.it));
    w.h = u / w.pairs;
    w.pair = u % w.pairs;
    w.unit = w.unit0 + u;
    w.rows = w.ntok * p.d.G - w.pair * 2 * kBM;
    w.it += w.n1 - w.n0;
    return true;
}

__device__ __forceinline__ bool page_ok(const SharedParams &p, int seq, int page, int *blk)
{
    const int b = __ldg(p.d.block_tables + (int64_t)seq * p.d.max_blocks + page);
    if (b < 0 || b >= p.d.num_blocks)
        return false;
    *blk = b;
    return true;
}

__global__ void __launch_bounds__(kSharedThreads, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ SharedParams p)
{
    extern __shared__ uint8_t smem_raw[];
    SharedSmem &sh = *reinterpret_cast<SharedSmem *>(align_smem_1024(smem_raw));
    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;

    if (tid == 32) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], 1);
            mbar_init(&sh.v_full[s], 1);
            mbar_init(&sh.v_empty[s], 1);
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.p_full[s], 4 * 32);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.o_empty[s], 4 * 32);
        }
        fence_barrier_init();
    }
    if (tid == 64) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the item space: warp 0 sums the groups and finds this CTA's first item ------
    if (warp == 0) {
        const bool ok = groups_ok(p, lane);
        SharedPlan *const plan = reinterpret_cast<SharedPlan *>(p.d.ws + p.plan_off);
        int64_t total = 0;
        int units = 0;
        for (int base = 0; ok && base < p.n_groups; base += 32) {
            SegWalk w{};
            w.g = base + lane;
            if (w.g < p.n_groups)
                load_group(p, w);
            int64_t n = (int64_t)w.pairs * p.d.Hkv * w.kt, incl = n;
            int un = w.pairs * p.d.Hkv, uincl = un;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
                const int b = __shfl_up_sync(0xffffffffu, uincl, o);
                if (lane >= o) {
                    incl += a;
                    uincl += b;
                }
            }
            if (blockIdx.x == 0 && w.g < p.n_groups) {
                SharedGroup &gp = plan->group[w.g];
                gp.item0 = total + incl - n;
                gp.unit0 = units + uincl - un;
                gp.pairs = w.pairs;
                gp.kt = w.kt;
                const int len = __ldg(p.shared_len + w.g);
                if (len < 0)
                    set_err(p.d.dev_err, HSA_DEVERR_BAD_LEN);
                if (len / kTileKeys > p.d.max_blocks)
                    set_err(p.d.dev_err, HSA_DEVERR_BAD_PAGE);
            }
            total += __shfl_sync(0xffffffffu, incl, 31);
            units += __shfl_sync(0xffffffffu, uincl, 31);
        }
        if (lane == 0)
            sh.N = total;
        const int64_t C = min(total, (int64_t)gridDim.x);
        if (blockIdx.x == 0 && lane == 0) {
            plan->N = total;
            plan->C = C;
            if (!ok)
                set_err(p.d.dev_err, HSA_DEVERR_BAD_LEN);
        }
        // second walk: the group that holds item i0
        const int64_t i0 = blockIdx.x < C ? (int64_t)blockIdx.x * total / C : total;
        total = 0;
        units = 0;
        for (int base = 0; ok && base < p.n_groups; base += 32) {
            SegWalk w{};
            w.g = base + lane;
            if (w.g < p.n_groups)
                load_group(p, w);
            int64_t n = (int64_t)w.pairs * p.d.Hkv * w.kt, incl = n;
            int un = w.pairs * p.d.Hkv, uincl = un;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t a = __shfl_up_sync(0xffffffffu, incl, o);
                const int b = __shfl_up_sync(0xffffffffu, uincl, o);
                if (lane >= o) {
                    incl += a;
                    uincl += b;
                }
            }
            if (total + incl - n <= i0 && i0 < total + incl) {
                sh.g0 = w.g;
                sh.unit0 = units + uincl - un;
                sh.item0 = total + incl - n;
            }
            total += __shfl_sync(0xffffffffu, incl, 31);
            units += __shfl_sync(0xffffffffu, uincl, 31);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int64_t N = sh.N;
    const int64_t C = min(N, (int64_t)gridDim.x);
    if ((int64_t)blockIdx.x >= C) {
        if (warp == 1)
            tmem_dealloc(sh.tmem_base, kTmemCols);
        return;
    }
    SegWalk w{};
    w.it = (int64_t)blockIdx.x * N / C;
    w.i1 = ((int64_t)blockIdx.x + 1) * N / C;
    w.item0 = sh.item0;
    w.g = sh.g0;
    w.unit0 = sh.unit0;
    load_group(p, w);
    const uint32_t tmem = sh.tmem_base;

    if (warp == 0) {
        // ================================================================ producer
        if (lane == 0) {
            const uint64_t pol_first = policy_evict_first(), pol_keep = policy_evict_last();
            bool ok = true;
            int kc = 0, sc = 0;
            while (ok && next_seg(p, w)) {
                const int nq = w.split() ? 1 : 2;
                if (!mbar_wait_sleep(&sh.q_empty, (sc & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&sh.q_full, nq * kOpBytes);
                const int tok0 = w.seq0 * p.d.T + w.pair * (2 * kBM / p.d.G);
                for (int t = 0; t < nq; ++t)
                    for (int hf = 0; hf < 2; ++hf)
                        tma_load_3d(sh.q[t] + hf * kHalfBytes, &tmQ, &sh.q_full, hf * 64,
                                    w.h * p.d.G, tok0 + t * (kBM / p.d.G), pol_keep);
                ++sc;
                // pages that more than one unit reads stay in L2
                const uint64_t pol = w.pairs > 1 ? pol_keep : pol_first;
                const int32_t *const table =
                    p.d.block_tables + (int64_t)w.seq0 * p.d.max_blocks;
                auto entry = [&](int page) { return page < w.pages ? __ldg(table + page) : 0; };
                int b0 = entry(2 * w.n0), b1 = entry(2 * w.n0 + 1);
                for (int n = w.n0; n < w.n1 && ok; ++n, ++kc) {
                    const int s = kc & 1;
                    const uint32_t ph = (kc >> 1) & 1;
                    // the next tile's block-table reads, ahead of the waits
                    int c0 = 0, c1 = 0;
                    if (n + 1 < w.n1) {
                        c0 = entry(2 * n + 2);
                        c1 = entry(2 * n + 3);
                    }
                    // an entry out of range: page 0 as a stand-in, masked below
                    if (b0 < 0 || b0 >= p.d.num_blocks || b1 < 0 || b1 >= p.d.num_blocks) {
                        set_err(p.d.dev_err, HSA_DEVERR_BAD_BLOCK);
                        b0 = b0 < 0 || b0 >= p.d.num_blocks ? 0 : b0;
                        b1 = b1 < 0 || b1 >= p.d.num_blocks ? 0 : b1;
                    }
                    if (2 * n + 1 >= w.pages)
                        b1 = b0;  // past the shared pages: loaded again, masked
                    for (int kv = 0; kv < 2; ++kv) {
                        if (!mbar_wait_sleep(kv ? &sh.v_empty[s] : &sh.k_empty[s], ph ^ 1)) {
                            ok = false;
                            break;
                        }
                        uint64_t *full = kv ? &sh.v_full[s] : &sh.k_full[s];
                        uint8_t *dst = kv ? sh.v[s] : sh.k[s];
                        const CUtensorMap *map = kv ? &tmV : &tmK;
                        mbar_arrive_expect_tx(full, kOpBytes);
                        for (int pg = 0; pg < 2; ++pg) {
                            const int32_t y = ((pg ? b1 : b0) * p.d.Hkv + w.h) * kTileKeys;
                            tma_load_2d(dst + pg * 8192, map, full, 0, y, pol);
                            tma_load_2d(dst + kHalfBytes + pg * 8192, map, full, 64, y, pol);
                        }
                    }
                    b0 = c0;
                    b1 = c1;
                }
            }
            if (!ok)
                set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
            // drain: no TMA write may still be in flight when the CTA exits
            for (int s = 0; s < 2 && kc > s; ++s) {
                const int last = s + ((kc - 1 - s) / 2) * 2;
                mbar_wait_sleep(&sh.k_full[s], (last >> 1) & 1);
                mbar_wait_sleep(&sh.v_full[s], (last >> 1) & 1);
            }
            if (sc > 0)
                mbar_wait_sleep(&sh.q_full, (sc - 1) & 1);
        }
    } else if (warp == 1) {
        // ================================================================ MMA issuer
        if (lane == 0) {
            const uint32_t id_s = idesc_bf16_f32(kBM, kBN, 0, 0);
            const uint32_t id_pv = idesc_bf16_f32(kBM, kD, 0, 1);
            const uint32_t dhi = smem_desc_sw128_hi(1024);
            const uint32_t q_lo[2] = {smem_desc_sw128_lo(smem_u32(sh.q[0]), 16),
                                      smem_desc_sw128_lo(smem_u32(sh.q[1]), 16)};
            const uint32_t k_lo[2] = {smem_desc_sw128_lo(smem_u32(sh.k[0]), 16),
                                      smem_desc_sw128_lo(smem_u32(sh.k[1]), 16)};
            const uint32_t v_lo[2] = {smem_desc_sw128_lo(smem_u32(sh.v[0]), kHalfBytes),
                                      smem_desc_sw128_lo(smem_u32(sh.v[1]), kHalfBytes)};
            // S_t = Q_q K^T of stage s; O_t (+)= P_t V of stage s, P_t in TMEM over S_t
            auto issue_s = [&](int t, int q, int s) {
                const uint32_t qa = q ? q_lo[1] : q_lo[0], kb = s ? k_lo[1] : k_lo[0];
                const uint32_t d = tmem + t * 128;
                tc_mma_ss_k<0>(d, desc_join(qa, dhi), desc_join(kb, dhi), id_s);
#pragma unroll
                for (int ks = 1; ks < kD / 16; ++ks) {
                    const uint32_t off = (ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2;
                    tc_mma_ss_k<1>(d, desc_join(qa + off, dhi), desc_join(kb + off, dhi), id_s);
                }
                tc_commit(&sh.s_full[t]);
            };
            auto issue_pv = [&](int t, int s, bool first) {
                const uint32_t vb = s ? v_lo[1] : v_lo[0];
                const uint32_t d = tmem + kColO + t * 128, a = tmem + t * 128;
                if (first)
                    tc_mma_ts_k<0>(d, a, desc_join(vb, dhi), id_pv);
                else
                    tc_mma_ts_k<1>(d, a, desc_join(vb, dhi), id_pv);
#pragma unroll
                for (int ks = 1; ks < kBN / 16; ++ks)
                    tc_mma_ts_k<1>(d, a + ks * 8, desc_join(vb + ks * (2048 >> 4), dhi), id_pv);
            };
            bool ok = true;
            int kc = 0, sc = 0;              // key tiles, segments so far
            int np[2] = {0, 0}, ns[2] = {0, 0};  // the same, of each query tile
            while (ok && next_seg(p, w)) {
                if (!mbar_wait_sleep(&sh.q_full, sc & 1) ||
                    !mbar_wait_sleep(&sh.k_full[kc & 1], (kc >> 1) & 1)) {
                    ok = false;
                    break;
                }
                ++sc;
                tc_fence_after();
                if (w.split()) {
                    // key tile j of the segment in region j % 2: S(j + 2) behind PV(j)
                    const int nn = w.n1 - w.n0;
                    issue_s(0, 0, kc & 1);
                    tc_commit(&sh.k_empty[kc & 1]);
                    if (nn > 1) {
                        if (!mbar_wait_sleep(&sh.k_full[(kc + 1) & 1], ((kc + 1) >> 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        issue_s(1, 0, (kc + 1) & 1);
                        tc_commit(&sh.k_empty[(kc + 1) & 1]);
                    }
                    if (nn <= 2)
                        tc_commit(&sh.q_empty);
                    for (int j = 0; j < nn && ok; j += 2) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (j + t >= nn || !ok)
                                continue;
                            const int s = kc & 1;
                            if (!mbar_wait_sleep(&sh.p_full[t], np[t] & 1) ||
                                !mbar_wait_sleep(&sh.v_full[s], (kc >> 1) & 1) ||
                                (j == 0 && !mbar_wait_sleep(&sh.o_empty[t], (ns[t] & 1) ^ 1))) {
                                ok = false;
                                continue;
                            }
                            ++np[t];
                            tc_fence_after();
                            issue_pv(t, s, j == 0);
                            tc_commit(&sh.v_empty[s]);
                            if (j + t + 2 < nn) {
                                if (!mbar_wait_sleep(&sh.k_full[s], ((kc + 2) >> 1) & 1)) {
                                    ok = false;
                                    continue;
                                }
                                tc_fence_after();
                                issue_s(t, 0, s);
                                tc_commit(&sh.k_empty[s]);
                                if (j + t + 3 == nn)
                                    tc_commit(&sh.q_empty);  // the segment's last S product
                            } else {
                                tc_commit(&sh.o_full[t]);
                            }
                            ++kc;
                        }
                    }
                    ++ns[0];
                    ns[1] += nn > 1;
                    continue;
                }
                issue_s(0, 0, kc & 1);
                issue_s(1, 1, kc & 1);
                tc_commit(&sh.k_empty[kc & 1]);
                if (w.n1 - w.n0 == 1)
                    tc_commit(&sh.q_empty);
                for (int n = w.n0; n < w.n1 && ok; ++n, ++kc) {
                    const int s = kc & 1;
                    const bool more = n + 1 < w.n1;
                    if (more && !mbar_wait_sleep(&sh.k_full[(kc + 1) & 1], ((kc + 1) >> 1) & 1)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (!ok)
                            continue;
                        if (!mbar_wait_sleep(&sh.p_full[t], np[t] & 1) ||
                            (t == 0 && !mbar_wait_sleep(&sh.v_full[s], (kc >> 1) & 1)) ||
                            (n == w.n0 && !mbar_wait_sleep(&sh.o_empty[t], (ns[t] & 1) ^ 1))) {
                            ok = false;
                            continue;
                        }
                        ++np[t];
                        tc_fence_after();
                        issue_pv(t, s, n == w.n0);
                        if (more)
                            issue_s(t, t, (kc + 1) & 1);
                        else
                            tc_commit(&sh.o_full[t]);
                    }
                    if (!ok)
                        break;
                    if (more)
                        tc_commit(&sh.k_empty[(kc + 1) & 1]);
                    if (n + 2 == w.n1)
                        tc_commit(&sh.q_empty);  // the segment's last S products are issued
                    tc_commit(&sh.v_empty[s]);
                }
                ++ns[0];
                ++ns[1];
            }
            if (ok) {
                // every MMA done before TMEM is released
#pragma unroll
                for (int t = 0; t < 2; ++t)
                    if (ok && ns[t] > 0)
                        ok = mbar_wait_sleep(&sh.o_full[t], (ns[t] - 1) & 1);
            }
            if (!ok)
                set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
        }
    } else {
        // ================================================================ softmax
        const int t = (warp - 2) >> 2;  // query tile: 0 = A (warps 2-5), 1 = B (warps 6-9)
        const int wq = warp & 3;
        const int row = wq * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t col_s = t * 128, col_o = kColO + t * 128;
        int np = 0, ns = 0;  // key tiles and segments of this query tile so far
        bool ok = true;
        while (ok && next_seg(p, w)) {
            const int step = w.split() ? 2 : 1;       // key tiles n0 + first, + step, ...
            const int first = w.split() ? t : 0;
            const int r = w.pair * 2 * kBM + (w.split() ? 0 : t * kBM) + row;  // of the group and head
            const bool row_ok = r < w.ntok * p.d.G;
            float *const oct = reinterpret_cast<float *>(p.d.ws + p.slot_off) +
                               ((int64_t)blockIdx.x + w.unit) * kSlotFloats +
                               (t * kBM + row) / 8 * kOctFloats;
            if (w.n0 + first >= w.n1) {  // one key tile, not this warpgroup's
                if (row_ok) {
                    oct[row & 7] = -INFINITY;
                    oct[8 + (row & 7)] = 0.f;
                }
                continue;
            }
            // a member may hold less than the shared pages
            int hi_row = 0;
            if (row_ok)
                hi_row = min(w.pages * kTileKeys,
                             clamp_len(__ldg(p.d.cached_len + w.seq0 + r / p.d.G / p.d.T)));
            float m_used = -INFINITY, l = 0.f;
            auto page_bits = [&](int n) -> int {
                int blk, bits = 0;
                if (2 * n < w.pages && page_ok(p, w.seq0, 2 * n, &blk))
                    bits |= 1;
                if (2 * n + 1 < w.pages && page_ok(p, w.seq0, 2 * n + 1, &blk))
                    bits |= 2;
                return bits;
            };
            int bits = page_bits(w.n0 + first);
            for (int n = w.n0 + first; n < w.n1; n += step, ++np) {
                const int next_bits = n + step < w.n1 ? page_bits(n + step) : 0;
                if (!mbar_wait_sleep(&sh.s_full[t], np & 1)) {
                    set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int hi = min(kBN, hi_row - n * kBN);
                const bool whole_tile = hi == kBN && bits == 3;
                // ---- the row's 128 scores: one TMEM read, kept in registers --------
                uint32_t r32[4][32];
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4)
                    tmem_ld32(lane_addr + col_s + c4 * 32, r32[c4]);
                tmem_wait_ld();
                if (!whole_tile) {
#pragma unroll
                    for (int c4 = 0; c4 < 4; ++c4)
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            if (c4 * 32 + c >= hi || !(bits & (c4 < 2 ? 1 : 2)))
                                r32[c4][c] = __float_as_uint(-INFINITY);
                }
                // ---- row max (three-input max, four chains) -----------------------
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4)
#pragma unroll
                    for (int c = 0; c < 32; c += 8) {
                        m4[0] = fmax3(m4[0], __uint_as_float(r32[c4][c + 0]), __uint_as_float(r32[c4][c + 1]));
                        m4[1] = fmax3(m4[1], __uint_as_float(r32[c4][c + 2]), __uint_as_float(r32[c4][c + 3]));
                        m4[2] = fmax3(m4[2], __uint_as_float(r32[c4][c + 4]), __uint_as_float(r32[c4][c + 5]));
                        m4[3] = fmax3(m4[3], __uint_as_float(r32[c4][c + 6]), __uint_as_float(r32[c4][c + 7]));
                    }
                const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.d.scale_log2;
                // ---- running max, raised only when it grows by more than 2^8 -------
                float m_new = m_used;
                if (mx != -INFINITY && (m_used == -INFINITY || mx > m_used + kRescaleSlack))
                    m_new = mx;
                const bool resc = m_used != -INFINITY && m_new != m_used;
                const float alpha = resc ? fast_exp2(m_used - m_new) : 1.0f;
                m_used = m_new;
                const float base = m_used == -INFINITY ? 0.f : m_used;
                // ---- P = 2^(s scale log2e - m) as bf16 pairs over S -----------------
                // whole tiles: the row sum takes the unrounded P (128 keys: bf16's
                // rounding averages out); partial ones the rounded P that PV multiplies
                const uint64_t sc2 = f2_make(p.d.scale_log2, p.d.scale_log2);
                const uint64_t nb2 = f2_make(-base, -base);
                uint64_t acc2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
                float accr = 0.f;
#pragma unroll
                for (int c4 = 0; c4 < 4; ++c4) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c) {
                        const uint64_t x2 = f2_fma(f2_make(__uint_as_float(r32[c4][2 * c]),
                                                           __uint_as_float(r32[c4][2 * c + 1])),
                                                   sc2, nb2);
                        float x0, x1;
                        f2_split(x2, x0, x1);
                        const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
                        pk[c] = pack_bf16(p0, p1);
                        if (whole_tile)
                            acc2[c & 1] = f2_add(acc2[c & 1], f2_make(p0, p1));
                        else
                            accr += bf16_lo(pk[c]) + bf16_hi(pk[c]);
                    }
                    tmem_st16(lane_addr + col_s + c4 * 16, pk);
                }
                // O (read by PV of this tile, which waits for this warp) is rescaled once
                // the score registers are free; the segment's first PV overwrites it
                if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; ++c4) {
                        uint32_t o32[32];
                        tmem_ld32(lane_addr + col_o + c4 * 32, o32);
                        tmem_wait_ld();
#pragma unroll
                        for (int c = 0; c < 32; ++c)
                            o32[c] = __float_as_uint(__uint_as_float(o32[c]) * alpha);
                        tmem_st32(lane_addr + col_o + c4 * 32, o32);
                    }
                }
                {
                    float a0, a1;
                    f2_split(f2_add(acc2[0], acc2[1]), a0, a1);
                    l = l * alpha + ((a0 + a1) + accr);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sh.p_full[t]);
                bits = next_bits;
            }
            if (!ok)
                break;
            // ---- the segment's state -----------------------------------------------
            if (!mbar_wait_sleep(&sh.o_full[t], ns & 1)) {
                set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
                ok = false;
                break;
            }
            ++ns;
            tc_fence_after();
            float4 *const dst = reinterpret_cast<float4 *>(oct + 16) + (row & 7);
            if (row_ok) {
                oct[row & 7] = m_used;
                oct[8 + (row & 7)] = l;
            }
#pragma unroll 1
            for (int c4 = 0; c4 < 4; ++c4) {
                uint32_t o32[32];
                tmem_ld32(lane_addr + col_o + c4 * 32, o32);
                tmem_wait_ld();
                if (row_ok) {
#pragma unroll
                    for (int c = 0; c < 32; c += 4)
                        dst[(c4 * 8 + c / 4) * 8] =
                            make_float4(__uint_as_float(o32[c]), __uint_as_float(o32[c + 1]),
                                        __uint_as_float(o32[c + 2]), __uint_as_float(o32[c + 3]));
                }
            }
            tc_fence_before();
            mbar_arrive(&sh.o_empty[t]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// ------------------------------------------------------ pass 2: own pages and new tokens
//
// What a sequence holds past the shared pages is often short (a question on a document), so
// the work is cut over many small streams instead of CTAs: four groups of MT warps a CTA,
// each with a range of 32-key items, a ring of stages and softmax states of its own, which
// loads its own tiles (lane 0, one item's stage refilled as it is done with) and writes its
// own state at the end of a (sequence, head) unit.  No barrier joins the groups, so one
// group's start and end of a unit hides under the others' tiles.  The T new tokens are the
// unit's last keys: their rows are written into the staged tile that they fall in.

constexpr int kKT = 32;                         // keys an item: half a page
constexpr int kGroups = 4;
constexpr int kDepth = 3;                       // stages a group
constexpr int kHalfTile = kKT * kD * 2;         // 8 KB: K or V of an item
constexpr int kItemBytes = 2 * kHalfTile;
constexpr int kInfoCap = 1024;                  // sequences whose lengths are kept in shared memory
constexpr int kOwnMaxThreads = kGroups * 2 * 32;

struct OwnSmem {
    alignas(1024) uint8_t stage[kGroups][kDepth][kItemBytes];  // [K lo|K hi|V lo|V hi]
    alignas(8) uint64_t full[kGroups][kDepth];
    alignas(8) uint64_t empty[kGroups][kDepth];  // MT = 2: the second warp is done with it
    int32_t ok[kGroups][kDepth];                 // the item's cached keys were loaded
    int2 info[kInfoCap];                         // (c, fp) of a sequence
    int32_t scan[kOwnMaxThreads];
    int32_t first_b[kGroups], first_before[kGroups];
    int32_t total_items, share;
};

// Position in a stream: sequence b, head h, item j of n; c cached tokens past the first
// page `fp` that is the sequence's own.
struct OwnWalk {
    int b, h, j, n, c, fp;
};

// c and fp of sequence b, from the inputs.
__device__ __forceinline__ int2 own_info(const SharedParams &p, bool share, int b)
{
    const int fp = share ? group_pages(p, group_of(p, b)) : 0;
    return make_int2(max(0, clamp_len(__ldg(p.d.cached_len + b)) - fp * kTileKeys), fp);
}

__device__ __forceinline__ int own_items(const SharedParams &p, int c)
{
    return (c + p.d.T + kKT - 1) / kKT;
}

__device__ __forceinline__ void own_load(const SharedParams &p, const OwnSmem &sh, OwnWalk &w)
{
    const int2 v = w.b < kInfoCap ? sh.info[w.b] : own_info(p, sh.share != 0, w.b);
    w.c = v.x;
    w.fp = v.y;
    w.n = own_items(p, w.c);
}

__device__ __forceinline__ void own_next(const SharedParams &p, const OwnSmem &sh, OwnWalk &w)
{
    if (++w.j == w.n) {
        w.j = 0;
        if (++w.h == p.d.Hkv) {
            w.h = 0;
            ++w.b;
            if (w.b < p.d.B)
                own_load(p, sh, w);
        }
    }
}

// Block-table entry of item w (-1: past the table); only read where it has cached keys.
__device__ __forceinline__ int own_entry(const SharedParams &p, const OwnWalk &w)
{
    const int page = w.fp + w.j / (kTileKeys / kKT);
    if (w.j * kKT >= w.c || page >= p.d.max_blocks)
        return -1;
    return __ldg(p.d.block_tables + (int64_t)w.b * p.d.max_blocks + page);
}

// Floats of an own segment's state: m[R], l[R], o[R][128] for R = G T rows, m and l padded
// to 16 bytes.
__host__ __device__ inline int own_pad(int rows) { return (rows + 3) & ~3; }
__host__ __device__ inline int own_slot_floats(int rows) { return 2 * own_pad(rows) + rows * kD; }

// MT: 16-row m-tiles of a sequence's G T query rows (1 or 2), a warp each.
template <int MT>
__global__ void __launch_bounds__(kGroups *MT * 32, 1)
    own_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ SharedParams p)
{
    extern __shared__ uint8_t smem_raw[];
    OwnSmem &sh = *reinterpret_cast<OwnSmem *>(align_smem_1024(smem_raw));
    constexpr int kThr = kGroups * MT * 32;
    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;
    const int grp = warp / MT, mt = warp % MT;
    const DecodeParams &d = p.d;

    if (tid == 0) {
        for (int i = 0; i < kGroups; ++i)
            for (int s = 0; s < kDepth; ++s) {
                mbar_init(&sh.full[i][s], 1);
                mbar_init(&sh.empty[i][s], 1);
            }
        fence_barrier_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    // Pass 1's CTAs signal only after their own wait, so everything queued before pass 1
    // has completed here: q, the new rows, lengths, tables and pool are final.  Nothing
    // here reads what pass 1 writes; the wait before the exit keeps pass 3 behind it.
    grid_launch_dependents();
    if (warp == 0) {
        const bool ok = groups_ok(p, lane);
        if (lane == 0)
            sh.share = ok;
    }
    __syncthreads();
    const bool share = sh.share != 0;

    // ---- items before each sequence; a stream an equal contiguous range ----------
    const int per = (d.B + kThr - 1) / kThr;
    const int b_lo = min(d.B, tid * per), b_hi = min(d.B, b_lo + per);
    {
        int local = 0;
        for (int b = b_lo; b < b_hi; ++b) {
            const int2 v = own_info(p, share, b);
            if (b < kInfoCap)
                sh.info[b] = v;
            local += own_items(p, v.x);
        }
        sh.scan[tid] = local;
        __syncthreads();
        if (warp == 0) {
            constexpr int kPer = kThr / 32;
            int v[kPer];
            int sum = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                v[j] = sh.scan[lane * kPer + j];
                sum += v[j];
            }
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += u;
            }
            int acc = incl - sum;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                sh.scan[lane * kPer + j] = acc;
                acc += v[j];
            }
            if (lane == 31)
                sh.total_items = incl;
        }
        __syncthreads();
    }
    const int64_t N = (int64_t)sh.total_items * d.Hkv;
    const int64_t C = min(N, (int64_t)gridDim.x * kGroups);
    // streams 0 .. gridDim - 1 on different CTAs: few items still use every SM
    const int64_t stream = (int64_t)grp * gridDim.x + blockIdx.x;
    const int64_t i0 = min(N, stream * N / C), i1 = min(N, (stream + 1) * N / C);
    {
        OwnPlan *const plan = reinterpret_cast<OwnPlan *>(d.ws + p.own_plan_off);
        int before = sh.scan[tid];
        for (int b = b_lo; b < b_hi; ++b) {
            const int n = own_items(p, b < kInfoCap ? sh.info[b].x : own_info(p, share, b).x);
#pragma unroll
            for (int i = 0; i < kGroups; ++i) {
                const int64_t at = min(N, ((int64_t)i * gridDim.x + blockIdx.x) * N / C);
                if ((int64_t)(before + n) * d.Hkv > at && (int64_t)before * d.Hkv <= at) {
                    sh.first_b[i] = b;
                    sh.first_before[i] = before;
                }
            }
            if (blockIdx.x == 0)  // for pass 3
                plan->before[b] = before;
            before += n;
        }
        if (blockIdx.x == 0 && tid == 0) {
            plan->N = N;
            plan->C = C;
        }
        __syncthreads();
    }
    if (i0 >= i1) {
        grid_dependency_wait();  // every CTA's exit stays ordered after pass 1
        return;
    }
    OwnWalk w;
    w.b = sh.first_b[grp];
    own_load(p, sh, w);
    {
        const int64_t off = i0 - (int64_t)sh.first_before[grp] * d.Hkv;
        w.h = (int)(off / w.n);
        w.j = (int)(off % w.n);
    }

    // ---- loads: item li of the stream, kDepth items ahead of the products ------------
    const uint64_t pol = policy_evict_first();
    OwnWalk lw = w;
    int64_t li = i0;
    int lst = 0;
    uint32_t lph = 0;  // parity of the stage's next empty phase (MT = 2)
    int entry = own_entry(p, lw);
    bool timed_out = false;
    auto load = [&](bool refill) {  // the group's first warp
        if (li >= i1)
            return;
        if (MT == 2 && refill && !timed_out && !mbar_wait(&sh.empty[grp][lst], lph)) {
            set_err(d.dev_err, HSA_DEVERR_TIMEOUT);
            timed_out = true;
        }
        if (lane == 0) {
            bool ok = lw.j * kKT < lw.c && !timed_out;
            if (ok && (entry < 0 || entry >= d.num_blocks)) {
                set_err(d.dev_err, lw.fp + lw.j / (kTileKeys / kKT) >= d.max_blocks
                                       ? HSA_DEVERR_BAD_PAGE
                                       : HSA_DEVERR_BAD_BLOCK);
                ok = false;
            }
            uint64_t *const full = &sh.full[grp][lst];
            sh.ok[grp][lst] = ok;
            if (ok) {
                uint8_t *const dst = sh.stage[grp][lst];
                const int32_t r = (entry * d.Hkv + lw.h) * kTileKeys + lw.j * kKT % kTileKeys;
                mbar_arrive_expect_tx(full, kItemBytes);
                tma_load_2d(dst, &tmK, full, 0, r, pol);
                tma_load_2d(dst + kHalfTile / 2, &tmK, full, 64, r, pol);
                tma_load_2d(dst + kHalfTile, &tmV, full, 0, r, pol);
                tma_load_2d(dst + kHalfTile + kHalfTile / 2, &tmV, full, 64, r, pol);
            } else {
                mbar_arrive(full);
            }
        }
        __syncwarp();
        ++li;
        if (li < i1) {
            own_next(p, sh, lw);
            entry = own_entry(p, lw);  // used at the next load
        }
        if (++lst == kDepth) {
            lst = 0;
            lph ^= refill ? 1 : 0;
        }
    };
    if (mt == 0)
        for (int i = 0; i < kDepth; ++i)
            load(false);

    // ---- products ---------------------------------------------------------------------
    const int g = lane >> 2, tq = lane & 3;
    const int q_r0 = mt * 16 + g, q_r1 = q_r0 + 8;
    const int t0 = q_r0 / d.G, t1 = q_r1 / d.G;
    const bool v0 = t0 < d.T, v1 = t1 < d.T;
    const int Hq = d.G * d.Hkv, rows = d.G * d.T;
    RowState st;
    uint32_t qa[kD / 16][4];
    int stg = 0;
    uint32_t ph = 0;
    bool fresh = true;
    for (int64_t i = i0; i < i1; ++i) {
        if (fresh) {
            fresh = false;
            st.m[0] = st.m[1] = -INFINITY;
            st.l[0] = st.l[1] = 0.f;
#pragma unroll
            for (int n = 0; n < kD / 8; ++n)
                st.o[n][0] = st.o[n][1] = st.o[n][2] = st.o[n][3] = 0.f;
            const __nv_bfloat16 *q0 =
                d.q + ((int64_t)(w.b * d.T + t0) * Hq + w.h * d.G + q_r0 % d.G) * kD;
            const __nv_bfloat16 *q1 =
                d.q + ((int64_t)(w.b * d.T + t1) * Hq + w.h * d.G + q_r1 % d.G) * kD;
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                const int c0 = ks * 16 + 2 * tq;
                qa[ks][0] = v0 ? __ldg(reinterpret_cast<const uint32_t *>(q0 + c0)) : 0u;
                qa[ks][1] = v1 ? __ldg(reinterpret_cast<const uint32_t *>(q1 + c0)) : 0u;
                qa[ks][2] = v0 ? __ldg(reinterpret_cast<const uint32_t *>(q0 + c0 + 8)) : 0u;
                qa[ks][3] = v1 ? __ldg(reinterpret_cast<const uint32_t *>(q1 + c0 + 8)) : 0u;
            }
        }
        if (!timed_out && !mbar_wait(&sh.full[grp][stg], ph)) {
            set_err(d.dev_err, HSA_DEVERR_TIMEOUT);
            timed_out = true;
        }
        uint8_t *const base = sh.stage[grp][stg];
        // keys 0 .. cached - 1 of the item are cached ones, key news + t is new token t
        const int news = w.c - w.j * kKT;
        const int cached = !timed_out && sh.ok[grp][stg] ? min(kKT, news) : 0;
        if (cached < kKT) {
            // the new tokens' rows; V rows of no key may hold anything, and 0 x NaN is NaN:
            // they become 0 (their scores are masked).  Both warps of a pair write the same.
            for (int e = lane; e < (kKT - cached) * (kD / 8); e += 32) {
                const int key = cached + e / (kD / 8), col = (e % (kD / 8)) * 8, t = key - news;
                uint4 vv = make_uint4(0, 0, 0, 0);
                uint8_t *const at = base + swz128_offset(key, col, kKT);
                if (t >= 0 && t < d.T) {
                    const int64_t src = ((int64_t)(w.b * d.T + t) * d.Hkv + w.h) * kD + col;
                    vv = __ldg(reinterpret_cast<const uint4 *>(d.v_new + src));
                    *reinterpret_cast<uint4 *>(at) = __ldg(reinterpret_cast<const uint4 *>(d.k_new + src));
                }
                *reinterpret_cast<uint4 *>(at + kHalfTile) = vv;
            }
            fence_proxy_async_smem();  // before the stage's next TMA write
            __syncwarp();
        }
        {
            const int T = d.T;
            auto vis = [&](int rr, int key) -> bool {
                const int t = rr == g ? t0 : t1;
                return t < T && (key < cached || (key >= news && key - news <= t));
            };
            const uint32_t sK = smem_u32(base);
            run_tile<kKT / 8>(st, qa, sK, sK + kHalfTile, kKT, 0, d.scale_log2, cached == kKT, v0, v1, vis);
        }
        __syncwarp();
        if (MT == 2 && mt == 1 && lane == 0)
            mbar_arrive(&sh.empty[grp][stg]);
        if (mt == 0)
            load(true);
        if (++stg == kDepth) {
            stg = 0;
            ph ^= 1;
        }
        const bool last = w.j == w.n - 1 || i == i1 - 1;
        if (last) {
            // ---- the segment's state, from the registers ------------------------------
            fresh = true;
            float l0 = st.l[0], l1 = st.l[1];
            l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
            l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
            l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
            const int pad = own_pad(rows);
            float *const part = reinterpret_cast<float *>(d.ws + p.own_off) +
                                (stream + w.b * d.Hkv + w.h) * own_slot_floats(rows);
            if (tq == 0) {
                if (v0) {
                    part[q_r0] = st.m[0];
                    part[pad + q_r0] = l0;
                }
                if (v1) {
                    part[q_r1] = st.m[1];
                    part[pad + q_r1] = l1;
                }
            }
            float *const o0 = part + 2 * pad + q_r0 * kD + 2 * tq;
#pragma unroll
            for (int n = 0; n < kD / 8; ++n) {
                if (v0)
                    *reinterpret_cast<float2 *>(o0 + n * 8) = make_float2(st.o[n][0], st.o[n][1]);
                if (v1)
                    *reinterpret_cast<float2 *>(o0 + 8 * kD + n * 8) =
                        make_float2(st.o[n][2], st.o[n][3]);
            }
        }
        own_next(p, sh, w);
    }
    grid_dependency_wait();
}

// ---------------------------------------------------------------- pass 3: merge, append

constexpr int kMergeThreads = 256;  // eight rows x 32 pieces of four dimensions
constexpr int kMergeBatch = 8;      // states whose loads are in flight together

__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const __grid_constant__ SharedParams p)
{
    const DecodeParams &d = p.d;
    const int tid = threadIdx.x;
    const int RT = d.G * d.T, Hq = d.G * d.Hkv;
    const int64_t rows = (int64_t)d.B * RT;
    const int h = blockIdx.x % d.Hkv;
    const int64_t r = (int64_t)(blockIdx.x / d.Hkv) * 8 + (tid & 7);
    const int d4 = tid >> 3;
    const bool on = r < rows;
    grid_launch_dependents();
    // inputs, final since before pass 1
    const int b = on ? (int)(r / RT) : 0, rr = (int)(r % RT);
    const int g = group_of(p, b);
    const int seq0 = __ldg(p.cu_group + g), seq1 = __ldg(p.cu_group + g + 1);
    grid_dependency_wait();

    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // n states at m (l at m + l_at, o at m + o_at), `step` floats apart
    auto take = [&](const float *m0, int l_at, int o_at, int64_t step, int n) {
        for (int c0 = 0; c0 < n; c0 += kMergeBatch) {
            float m[kMergeBatch], l[kMergeBatch];
            float4 x[kMergeBatch];
#pragma unroll
            for (int i = 0; i < kMergeBatch; ++i) {
                m[i] = -INFINITY;
                l[i] = 0.f;
                x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c0 + i < n) {
                    const float *s = m0 + (c0 + i) * step;
                    m[i] = __ldcg(s);
                    l[i] = __ldcg(s + l_at);
                    x[i] = __ldcg(reinterpret_cast<const float4 *>(s + o_at));
                }
            }
            float M1 = M;
#pragma unroll
            for (int i = 0; i < kMergeBatch; ++i)
                M1 = fmaxf(M1, m[i]);
            if (M1 == -INFINITY)
                continue;
            const float a = fast_exp2(M - M1);
            M = M1;
            L *= a;
            o.x *= a;
            o.y *= a;
            o.z *= a;
            o.w *= a;
#pragma unroll
            for (int i = 0; i < kMergeBatch; ++i) {
                if (m[i] == -INFINITY)
                    continue;  // a state of no keys: its o was not written
                const float f = fast_exp2(m[i] - M1);
                L += l[i] * f;
                o.x += x[i].x * f;
                o.y += x[i].y * f;
                o.z += x[i].z * f;
                o.w += x[i].w * f;
            }
        }
    };
    if (on) {
        const OwnPlan *const own = reinterpret_cast<const OwnPlan *>(d.ws + p.own_plan_off);
        const SharedPlan *const plan = reinterpret_cast<const SharedPlan *>(d.ws + p.plan_off);
        const SharedGroup *const gp = &plan->group[g];
        const int64_t oN = __ldcg(&own->N), oC = __ldcg(&own->C);
        const int before = __ldcg(&own->before[b]);
        const int next = b + 1 < d.B ? __ldcg(&own->before[b + 1]) : (int)(oN / d.Hkv);
        const int64_t N = __ldcg(&plan->N), C = __ldcg(&plan->C);
        const int64_t item0 = __ldcg(&gp->item0);
        const int unit0 = __ldcg(&gp->unit0), pairs = __ldcg(&gp->pairs), kt = __ldcg(&gp->kt);
        // the sequence's own states: streams c_lo .. c_hi of pass 2
        {
            const int n = next - before;
            const int64_t s0 = (int64_t)before * d.Hkv + (int64_t)h * n;
            const int64_t c_lo = ((s0 + 1) * oC - 1) / oN, c_hi = ((s0 + n) * oC - 1) / oN;
            const int step = own_slot_floats(RT), pad = own_pad(RT);
            const float *s = reinterpret_cast<const float *>(d.ws + p.own_off) +
                             (c_lo + b * d.Hkv + h) * step;
            take(s + rr, pad, 2 * pad - rr + rr * kD + 4 * d4, step, (int)(c_hi - c_lo) + 1);
        }
        // the shared segments' states
        if (N > 0 && kt > 0) {
            const int64_t rg = r - (int64_t)seq0 * RT;  // row of the group
            const int pair = (int)(rg / (2 * kBM)), row = (int)(rg % (2 * kBM));
            const int un = h * pairs + pair;
            const int64_t s0 = item0 + (int64_t)un * kt;
            const int64_t c_lo = ((s0 + 1) * C - 1) / N, c_hi = ((s0 + kt) * C - 1) / N;
            const float *s = reinterpret_cast<const float *>(d.ws + p.slot_off) +
                             (c_lo + unit0 + un) * kSlotFloats + row / 8 * kOctFloats + (row & 7);
            const int n = (int)(c_hi - c_lo) + 1;
            const int o_at = 16 - (row & 7) + (d4 * 8 + (row & 7)) * 4;
            // a unit of one query tile left two states a row, 128 rows apart
            const bool split = (int64_t)(seq1 - seq0) * RT - (int64_t)pair * 2 * kBM <= kBM;
            if (split)
                take(s, 8, o_at, kSlotFloats / 2, 2 * n);
            else
                take(s, 8, o_at, kSlotFloats, n);
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int t = rr / d.G, hh = rr % d.G;
        *reinterpret_cast<uint2 *>(d.out + ((int64_t)(b * d.T + t) * Hq + h * d.G + hh) * kD + 4 * d4) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    }
    if (d.flags & kDecodeAppend) {
        // every read of the pool is done: the new rows, one 16-byte chunk of K and V a thread
        const int64_t chunks = (int64_t)d.B * d.T * d.Hkv * (kD / 8);
        for (int64_t e = (int64_t)blockIdx.x * kMergeThreads + tid; e < chunks;
             e += (int64_t)gridDim.x * kMergeThreads) {
            const int ch = (int)(e % (kD / 8));
            const int64_t th = e / (kD / 8);
            const int hk = (int)(th % d.Hkv);
            const int64_t bt = th / d.Hkv;
            const int sb = (int)(bt / d.T);
            const int64_t pos = (int64_t)clamp_len(__ldg(d.cached_len + sb)) + bt % d.T;
            if (pos / kTileKeys >= d.max_blocks) {
                set_err(d.dev_err, HSA_DEVERR_BAD_PAGE);
                continue;
            }
            int blk = 0;
            if (!page_ok(p, sb, (int)(pos / kTileKeys), &blk)) {
                set_err(d.dev_err, HSA_DEVERR_BAD_BLOCK);
                continue;
            }
            const int64_t to = (((int64_t)blk * d.Hkv + hk) * kTileKeys + pos % kTileKeys) * (kD / 8) + ch;
            d.k_dst[to] = __ldg(reinterpret_cast<const uint4 *>(d.k_new) + e);
            d.v_dst[to] = __ldg(reinterpret_cast<const uint4 *>(d.v_new) + e);
        }
    }
}

template <typename... Args>
cudaError_t launch_dependent(void (*kern)(Args...), unsigned grid, unsigned threads, size_t smem,
                             cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

size_t pad256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace

SharedLayout shared_layout(size_t start, int ctas, int B, int T, int G, int Hkv, int n_groups)
{
    SharedLayout l;
    l.plan = pad256(start);
    l.own_plan = l.plan + pad256(sizeof(SharedPlan) + (size_t)n_groups * sizeof(SharedGroup));
    l.slots = l.own_plan + pad256(sizeof(OwnPlan) + (size_t)B * sizeof(int32_t));
    // segments in order move on by a CTA, a unit or both, so (CTA, unit)'s slot is
    // CTA + unit; units of pass 1: 256 rows of a group and a KV head
    const size_t units = ((size_t)B * T * G / (2 * kBM) + (n_groups < B ? n_groups : B)) * Hkv;
    l.own = l.slots + pad256((ctas + units) * kSlotFloats * sizeof(float));
    l.total = l.own + ((size_t)ctas * kGroups + (size_t)B * Hkv) * own_slot_floats(G * T) * sizeof(float);
    return l;
}

cudaError_t launch_shared(const CUtensorMap &tmK, const CUtensorMap &tmV, const CUtensorMap &tmQ,
                          const CUtensorMap &tmK32, const CUtensorMap &tmV32,
                          const SharedParams &p, int ctas, cudaStream_t stream)
{
    const size_t smem1 = sizeof(SharedSmem) + 1024, smem2 = sizeof(OwnSmem) + 1024;
    const int MT = (p.d.G * p.d.T + 15) / 16;
    auto own = MT == 1 ? own_kernel<1> : own_kernel<2>;
    // the opt-in shared-memory sizes are set once per process
    static bool attr_set[3] = {false, false, false};
    if (!attr_set[0]) {
        const cudaError_t e = cudaFuncSetAttribute(
            shared_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem1);
        if (e != cudaSuccess)
            return e;
        attr_set[0] = true;
    }
    if (!attr_set[MT]) {
        const cudaError_t e =
            cudaFuncSetAttribute(own, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem2);
        if (e != cudaSuccess)
            return e;
        attr_set[MT] = true;
    }
    cudaError_t e = launch_dependent(shared_kernel, (unsigned)ctas, kSharedThreads, smem1, stream,
                                     tmK, tmV, tmQ, p);
    if (e == cudaSuccess)
        e = launch_dependent(own, (unsigned)ctas, kGroups * MT * 32, smem2, stream, tmK32, tmV32, p);
    if (e == cudaSuccess) {
        const int64_t octs = ((int64_t)p.d.B * p.d.G * p.d.T + 7) / 8;
        e = launch_dependent(merge_kernel, (unsigned)(octs * p.d.Hkv), kMergeThreads, 0, stream, p);
    }
    return e;
}

}  // namespace hsa
