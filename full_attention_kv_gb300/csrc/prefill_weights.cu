// prefill_weights.cu -- the weight that a prompt's last queries put on every cached key (sm_103a).
//
// What it computes: for request r with n tokens in the pool, KV head h, and its last T queries of
// G heads each (row = t G + hh, at position n - T + t),
//   s[row][j] = scale q.k_j (j <= n - T + t),  lse[row] = log sum_j exp s,
//   w[j] = decay w_prev[j] + sum over rows of exp(s[row][j] - lse[row]).
// The sum over rows needs every row's lse first, and G T rows of scores (up to 2 KB a key) cost
// more to keep than a key's 256 bytes cost to read again: two passes over K, each S on tcgen05.
//
// Pass 1 takes the rows as TMEM lanes (S = Q K^T, 128 rows x 128 keys): a thread owns a row, keeps
// its running maximum and sum over the keys, and leaves them in the workspace.  Pass 2 takes the
// keys as lanes (S^T = K Q^T, the same tiles in shared memory with A and B exchanged): a thread
// owns a key, and the sum over rows is its own.  Neither sums across threads.
//
// Both: persistent, one CTA an SM; the 128-key tiles (two pages) of all (request, KV head) units
// laid end to end and cut into equal ranges.  Warp 0 loads Q (up to four tiles of 128 rows) at a
// unit's start and streams K; one thread of warp 1 issues the MMAs into four TMEM slots of 128
// columns, two a warpgroup; warps 2-5 and 6-9 are the two warpgroups, which take a unit's row
// tiles in turn (pass 1; key tiles in turn where there is one row tile) or key tiles (pass 2).
// The states of a unit's CTAs lie side by side, and their order is fixed: so are the sums.
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

constexpr int kD = 128;
constexpr int kBlock = 128;                // rows or keys of a tile
constexpr int kHalfBytes = kBlock * 128;   // 128 rows x 64 bf16 (one swizzle column block)
constexpr int kTileBytes = 2 * kHalfBytes; // 32 KB
constexpr int kTiles = 6;                  // Q tiles and K stages together
constexpr int kMaxStages = 4;
constexpr int kMaxRowTiles = 4;
constexpr int kThreads = 320;
constexpr uint32_t kTmemCols = 512;
constexpr float kSlack = 8.0f;             // a running maximum may lag by so much (log2 units)

struct alignas(1024) PromptSmem {
    uint8_t tile[kTiles][kTileBytes];
    alignas(16) float neg_lse[2][kMaxRowTiles * kBlock];  // pass 2: a copy a warpgroup
    alignas(8) uint64_t q_full, q_empty, done;
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];
    uint64_t s_full[4], s_empty[4];
    int32_t scan[kThreads];
    int32_t first_r, before, total;
    uint32_t tmem_base;
};

struct Request {
    int n, m, T, seq, row0;  // tokens, new rows, queries, sequence, first query row; T = 0: left out
};

__device__ __forceinline__ Request request(const PromptParams &p, int r, int *err)
{
    Request q{0, 0, 0, 0, 0};
    const int c0 = __ldg(p.cu_rows + r), c1 = __ldg(p.cu_rows + r + 1);
    const int n = __ldg(p.kv_len + r), seq = __ldg(p.seq_idx + r);
    if (c0 < 0 || c1 < c0 || c1 > p.rows) {
        *err = HSA_DEVERR_BAD_LEN;
        return q;
    }
    if (c1 == c0)
        return q;
    if (seq < 0 || seq >= p.batch) {
        *err = HSA_DEVERR_BAD_SEQ;
        return q;
    }
    if (n < c1 - c0 || n > p.w_stride) {
        *err = HSA_DEVERR_BAD_LEN;
        return q;
    }
    q.n = n;
    q.m = c1 - c0;
    q.T = min(p.window, q.m);
    q.seq = seq;
    q.row0 = c1 - q.T;
    return q;
}

__device__ __forceinline__ int tiles_of(const Request &q) { return q.T > 0 ? (q.n + kBlock - 1) / kBlock : 0; }

// Pool row of page `page` of head h, or -1: past the tokens (not loaded, masked by position), or
// out of reach (flagged).
__device__ __forceinline__ int64_t page_row(const PromptParams &p, const Request &q, int h, int page, bool report)
{
    if ((int64_t)page * 64 >= q.n)
        return -1;
    if (page >= p.max_blocks) {
        if (report)
            set_err(p.dev_err, HSA_DEVERR_BAD_PAGE);
        return -1;
    }
    const int blk = __ldg(p.block_tables + (int64_t)q.seq * p.max_blocks + page);
    if (blk < 0 || blk >= p.num_blocks) {
        if (report)
            set_err(p.dev_err, HSA_DEVERR_BAD_BLOCK);
        return -1;
    }
    return ((int64_t)blk * p.Hkv + h) * 64;
}

struct Walk {
    int r, h, j, nt;  // request, KV head, key tile j of nt
    Request q;
};

template <int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ,
                  const PromptParams p, const int q_tiles, const int stages)
{
    extern __shared__ uint8_t smem_raw[];
    PromptSmem &sh = *reinterpret_cast<PromptSmem *>(align_smem_1024(smem_raw));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- this CTA's contiguous range of key tiles ------------------------------------------
    const int per = (p.R + kThreads - 1) / kThreads;
    const int r_lo = min(p.R, tid * per), r_hi = min(p.R, r_lo + per);
    int local = 0;
    for (int r = r_lo; r < r_hi; ++r) {
        int err = 0;
        local += tiles_of(request(p, r, &err));
        if (PASS == 1 && err && blockIdx.x == 0)
            set_err(p.dev_err, err);
    }
    sh.scan[tid] = local;
    __syncthreads();
    if (warp == 0) {
        constexpr int kPer = kThreads / 32;
        int v[kPer], sum = 0;
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
            sh.total = incl;
    }
    __syncthreads();
    const int64_t N = (int64_t)sh.total * p.Hkv;
    const int64_t C = N < (int64_t)gridDim.x ? N : (int64_t)gridDim.x;
    if ((int64_t)blockIdx.x >= C)
        return;
    const int64_t i0 = (int64_t)blockIdx.x * N / C, i1 = ((int64_t)blockIdx.x + 1) * N / C;
    {
        int before = sh.scan[tid], err = 0;
        for (int r = r_lo; r < r_hi; ++r) {
            const int nt = tiles_of(request(p, r, &err));
            if ((int64_t)(before + nt) * p.Hkv > i0 && (int64_t)before * p.Hkv <= i0) {
                sh.first_r = r;
                sh.before = before;
            }
            before += nt;
        }
    }
    if (tid == 0) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 1);
        mbar_init(&sh.done, 1);
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], 1);
        }
        for (int s = 0; s < 4; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.s_empty[s], kBlock);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;

    Walk w;
    int err_unused = 0;
    w.r = sh.first_r;
    w.q = request(p, w.r, &err_unused);
    w.nt = tiles_of(w.q);
    {
        const int64_t off = i0 - (int64_t)sh.before * p.Hkv;
        w.h = (int)(off / w.nt);
        w.j = (int)(off % w.nt);
    }
    auto next_unit = [&](Walk &x) {  // after a unit's last tile
        x.j = 0;
        if (++x.h < p.Hkv)
            return;
        x.h = 0;
        do {
            if (++x.r >= p.R)
                return;
            x.q = request(p, x.r, &err_unused);
            x.nt = tiles_of(x.q);
        } while (x.nt == 0);
    };
    auto row_tiles = [&](const Walk &x) { return (x.q.T * p.G + kBlock - 1) / kBlock; };

    if (warp == 0) {
        // ------------------------------------------------------------------------ producer
        const uint64_t pol = policy_evict_first();
        int64_t k = 0;       // key tiles issued
        int units = 0;
        bool ok = true;
        for (int64_t i = i0; i < i1 && ok; ++units) {
            const int64_t end = i + min((int64_t)(w.nt - w.j), i1 - i);
            const int nq = row_tiles(w);
            if (lane == 0) {
                if (units > 0 && !mbar_wait_sleep(&sh.q_empty, (uint32_t)(units - 1) & 1)) {
                    ok = false;
                } else {
                    mbar_arrive_expect_tx(&sh.q_full, nq * kTileBytes);
                    for (int t = 0; t < nq; ++t) {
                        const int row = w.q.row0 + t * (kBlock / p.G);
                        tma_load_3d(sh.tile[t], &tmQ, &sh.q_full, 0, w.h * p.G, row, pol);
                        tma_load_3d(sh.tile[t] + kHalfBytes, &tmQ, &sh.q_full, 64, w.h * p.G, row, pol);
                    }
                }
            }
            // pool rows of 32 pages (16 tiles) at a time, a lane each, a batch ahead
            int j = w.j, batch = w.j;
            int64_t cur = page_row(p, w.q, w.h, 2 * batch + lane, PASS == 1);
            int64_t nxt = page_row(p, w.q, w.h, 2 * batch + 32 + lane, PASS == 1);
            for (; i < end; ++i, ++j, ++k) {
                if (j - batch == 16) {
                    batch = j;
                    cur = nxt;
                    nxt = page_row(p, w.q, w.h, 2 * batch + 32 + lane, PASS == 1);
                }
                const int64_t y0 = __shfl_sync(0xffffffffu, cur, 2 * (j - batch));
                const int64_t y1 = __shfl_sync(0xffffffffu, cur, 2 * (j - batch) + 1);
                if (lane == 0 && ok) {
                    const int st = (int)(k % stages);
                    if (!mbar_wait_sleep(&sh.k_empty[st], (uint32_t)((k / stages) & 1) ^ 1)) {
                        ok = false;
                    } else {
                        uint8_t *dst = sh.tile[q_tiles + st];
                        const int pages = (y0 >= 0) + (y1 >= 0);
                        if (pages == 0)
                            mbar_arrive(&sh.k_full[st]);
                        else
                            mbar_arrive_expect_tx(&sh.k_full[st], pages * (kTileBytes / 2));
                        if (y0 >= 0) {
                            tma_load_2d(dst, &tmK, &sh.k_full[st], 0, (int32_t)y0, pol);
                            tma_load_2d(dst + kHalfBytes, &tmK, &sh.k_full[st], 64, (int32_t)y0, pol);
                        }
                        if (y1 >= 0) {
                            tma_load_2d(dst + 8192, &tmK, &sh.k_full[st], 0, (int32_t)y1, pol);
                            tma_load_2d(dst + kHalfBytes + 8192, &tmK, &sh.k_full[st], 64, (int32_t)y1, pol);
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok)
                    break;
            }
            next_unit(w);
        }
        if (lane == 0) {
            if (!ok)
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
            // no copy may still be in flight when the CTA exits
            for (int64_t s = 0; s < stages && s < k; ++s) {
                const int64_t last = s + ((k - 1 - s) / stages) * stages;
                mbar_wait_sleep(&sh.k_full[s], (uint32_t)((last / stages) & 1));
            }
            if (units > 0)
                mbar_wait_sleep(&sh.q_full, (uint32_t)(units - 1) & 1);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            const uint32_t dhi = smem_desc_sw128_hi(1024);
            int64_t k = 0;
            int units = 0;
            uint32_t cnt0 = 0, cnt1 = 0;  // tiles handed to each warpgroup
            bool ok = true;
            for (int64_t i = i0; i < i1 && ok; ++units) {
                const int64_t end = i + min((int64_t)(w.nt - w.j), i1 - i);
                const int nq = row_tiles(w), rows = w.q.T * p.G;
                ok = mbar_wait_sleep(&sh.q_full, (uint32_t)units & 1);
                for (; i < end && ok; ++i, ++k) {
                    const int st = (int)(k % stages);
                    if (!(ok = mbar_wait_sleep(&sh.k_full[st], (uint32_t)((k / stages) & 1))))
                        break;
                    tc_fence_after();
                    const uint32_t kl = smem_desc_sw128_lo(smem_u32(sh.tile[q_tiles + st]), 16);
                    for (int t = 0; t < nq; ++t) {
                        const int wg = PASS == 2 || nq == 1 ? (int)(k & 1) : t & 1;
                        const uint32_t c = wg ? cnt1++ : cnt0++;
                        const int slot = 2 * wg + (c & 1);
                        if (!(ok = mbar_wait_sleep(&sh.s_empty[slot], ((c >> 1) & 1) ^ 1)))
                            break;
                        tc_fence_after();
                        const uint32_t ql = smem_desc_sw128_lo(smem_u32(sh.tile[t]), 16);
                        const int cols = PASS == 1 ? kBlock : min(kBlock, (rows - t * kBlock + 15) & ~15);
                        const uint32_t id = idesc_bf16_f32(kBlock, cols, 0, 0);
                        const uint32_t a = PASS == 1 ? ql : kl, b = PASS == 1 ? kl : ql;
                        const uint32_t d = tmem + slot * kBlock;
                        tc_mma_ss_k<0>(d, desc_join(a, dhi), desc_join(b, dhi), id);
#pragma unroll
                        for (int ks = 1; ks < kD / 16; ++ks) {
                            const uint32_t off = (ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2;
                            tc_mma_ss_k<1>(d, desc_join(a + off, dhi), desc_join(b + off, dhi), id);
                        }
                        tc_commit(&sh.s_full[slot]);
                    }
                    if (ok)
                        tc_commit(&sh.k_empty[st]);
                }
                if (ok)
                    tc_commit(&sh.q_empty);
                next_unit(w);
            }
            if (!ok)
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
            tc_commit(&sh.done);  // every MMA done before TMEM is released
            mbar_wait_sleep(&sh.done, 0);
        }
    } else {
        // ------------------------------------------------------------- rows' or keys' threads
        const int wg = (warp - 2) >> 2, wq = warp & 3;
        const int me = wq * 32 + lane;  // TMEM lane
        const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
        const uint64_t sc2 = f2_make(p.scale_log2, p.scale_log2);
        const int row_cap = q_tiles * kBlock;
        uint32_t cnt = 0;
        int64_t k = 0;
        bool ok = true;
        // bit e: page 2 batch + e can be read
        auto pages_ok = [&](int batch) {
            const int page = 2 * batch + lane;
            return __ballot_sync(0xffffffffu, (int64_t)page * 64 >= w.q.n || page_row(p, w.q, w.h, page, false) >= 0);
        };
        // the next TMEM slot of this warpgroup.  After a wait that gave up no further one is
        // made, but every tile is walked through: the warpgroup's barriers count on all of it.
        auto take = [&]() -> uint32_t {
            const uint32_t slot = 2 * wg + (cnt & 1);
            if (ok && !mbar_wait_sleep(&sh.s_full[slot], (cnt >> 1) & 1)) {
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
                ok = false;
            }
            __syncwarp();
            tc_fence_after();
            return slot;
        };
        auto give = [&](uint32_t slot) {
            tc_fence_before();
            mbar_arrive(&sh.s_empty[slot]);
            ++cnt;
        };
        for (int64_t i = i0; i < i1;) {
            const int64_t unit = (int64_t)w.r * p.Hkv + w.h;
            const int64_t end = i + min((int64_t)(w.nt - w.j), i1 - i);
            const int nq = row_tiles(w), n = w.q.n, T = w.q.T, rows = T * p.G;
            int j = w.j, batch = w.j;
            uint32_t good = pages_ok(batch);
            if constexpr (PASS == 1) {
                // the sums with what their roundings lost (a row has up to a million terms)
                float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lost[2] = {0.f, 0.f};
                for (; i < end; ++i, ++j, ++k) {
                    if (j - batch == 16) {
                        batch = j;
                        good = pages_ok(batch);
                    }
                    const uint32_t pair = good >> (2 * (j - batch)) & 3u;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = nq == 1 ? 0 : wg + 2 * e;
                        if (t >= nq || (nq == 1 && (e == 1 || (int)(k & 1) != wg)))
                            continue;
                        const uint32_t slot = take();
                        // keys of the tile this row sees: 0 .. hi - 1
                        const int hi = min(n, n - T + (t * kBlock + me) / p.G + 1) - j * kBlock;
                        const bool whole = __all_sync(0xffffffffu, hi >= kBlock) && pair == 3u;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint32_t x[2][32];
                            tmem_ld32(lane_addr + slot * kBlock + half * 64, x[0]);
                            tmem_ld32(lane_addr + slot * kBlock + half * 64 + 32, x[1]);
                            tmem_wait_ld();
                            if (half == 1)
                                give(slot);
                            if (!whole) {
                                const int top = (pair >> half & 1u) ? hi - half * 64 : 0;
#pragma unroll
                                for (int c = 0; c < 64; ++c)
                                    if (c >= top)
                                        x[c >> 5][c & 31] = __float_as_uint(-INFINITY);
                            }
                            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int c = 0; c < 64; c += 8)
#pragma unroll
                                for (int f = 0; f < 4; ++f)
                                    mx[f] = fmax3(mx[f], __uint_as_float(x[c >> 5][(c & 31) + 2 * f]),
                                                  __uint_as_float(x[c >> 5][(c & 31) + 2 * f + 1]));
                            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
                            if (top != -INFINITY && (m[e] == -INFINITY || top > m[e] + kSlack)) {
                                const float f = m[e] == -INFINITY ? 0.f : fast_exp2(m[e] - top);
                                l[e] *= f;
                                lost[e] *= f;
                                m[e] = top;
                            }
                            const float base = m[e] == -INFINITY ? 0.f : m[e];
                            const uint64_t nb2 = f2_make(-base, -base);
                            uint64_t acc[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll
                            for (int c = 0; c < 64; c += 2) {
                                float a, b;
                                f2_split(f2_fma(f2_make(__uint_as_float(x[c >> 5][c & 31]),
                                                        __uint_as_float(x[c >> 5][(c & 31) + 1])),
                                                sc2, nb2),
                                         a, b);
                                acc[c >> 1 & 1] = f2_add(acc[c >> 1 & 1], f2_make(fast_exp2(a), fast_exp2(b)));
                            }
                            float a, b;
                            f2_split(f2_add(acc[0], acc[1]), a, b);
                            const float add = (a + b) - lost[e], sum = l[e] + add;
                            lost[e] = (sum - l[e]) - add;
                            l[e] = sum;
                        }
                    }
                }
                // this CTA's part of the unit's rows (both warpgroups' where there is one row tile)
                float2 *const to = p.part + ((unit + blockIdx.x) * 2 + wg) * row_cap + me;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = nq == 1 ? 0 : wg + 2 * e;
                    if (t < nq && (nq > 1 || e == 0))
                        to[t * kBlock] = make_float2(m[e], l[e]);
                }
            } else {
                // ---- the rows' lse, out of the states of every CTA that met the unit ----------
                {
                    const int64_t u0 = i - w.j, u1 = u0 + w.nt;
                    const int64_t c_lo = ((u0 + 1) * C - 1) / N, c_hi = (u1 * C - 1) / N;
                    named_bar_sync(1 + wg, kBlock);  // the last unit's readers are done
                    for (int t = 0; t < nq; ++t) {
                        float M = -INFINITY, L = 0.f;
                        for (int64_t c = c_lo; c <= c_hi; ++c)
                            for (int g = nq == 1 ? 0 : t & 1; g <= (nq == 1 ? 1 : t & 1); ++g) {
                                const float2 s = __ldcg(p.part + ((unit + c) * 2 + g) * row_cap + t * kBlock + me);
                                const float top = fmaxf(M, s.x);
                                if (top != -INFINITY)
                                    L = L * fast_exp2(M - top) + s.y * fast_exp2(s.x - top);
                                M = top;
                            }
                        const bool on = t * kBlock + me < rows && L > 0.f;
                        sh.neg_lse[wg][t * kBlock + me] = on ? -(M + log2f(L)) : -INFINITY;
                    }
                    named_bar_sync(1 + wg, kBlock);
                }
                const int64_t at = ((int64_t)w.q.seq * p.Hkv + w.h) * p.w_stride;
                for (; i < end; ++i, ++j, ++k) {
                    if (j - batch == 16) {
                        batch = j;
                        good = pages_ok(batch);
                    }
                    if ((int)(k & 1) != wg)
                        continue;
                    const int pos = j * kBlock + me;
                    const int first = max(0, pos - (n - T)) * p.G;  // rows that see this key: first ..
                    const bool all = __all_sync(0xffffffffu, first == 0);
                    const float old = p.w_prev && pos < n - w.q.m ? p.w_prev[at + pos] : 0.f;
                    uint64_t acc[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
                    for (int t = 0; t < nq; ++t) {
                        const uint32_t slot = take();
                        const int top = min(kBlock, rows - t * kBlock);
                        for (int c0 = 0; c0 < top; c0 += 32) {
                            uint32_t x[32];
                            tmem_ld32(lane_addr + slot * kBlock + c0, x);
                            const float4 *const nl = reinterpret_cast<const float4 *>(&sh.neg_lse[wg][t * kBlock + c0]);
                            tmem_wait_ld();
                            if (all && c0 + 32 <= top) {
#pragma unroll
                                for (int c = 0; c < 32; c += 4) {
                                    const float4 y = nl[c >> 2];
                                    float a, b, d, e;
                                    f2_split(f2_fma(f2_make(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2,
                                                    f2_make(y.x, y.y)), a, b);
                                    f2_split(f2_fma(f2_make(__uint_as_float(x[c + 2]), __uint_as_float(x[c + 3])), sc2,
                                                    f2_make(y.z, y.w)), d, e);
                                    acc[0] = f2_add(acc[0], f2_make(fast_exp2(a), fast_exp2(b)));
                                    acc[1] = f2_add(acc[1], f2_make(fast_exp2(d), fast_exp2(e)));
                                }
                            } else {
#pragma unroll
                                for (int c = 0; c < 32; ++c) {
                                    const int row = t * kBlock + c0 + c;
                                    if (row >= first && row < rows) {
                                        const float a = fast_exp2(
                                            fmaf(__uint_as_float(x[c]), p.scale_log2, sh.neg_lse[wg][row]));
                                        acc[c & 1] = f2_add(acc[c & 1], f2_make(a, 0.f));
                                    }
                                }
                            }
                        }
                        give(slot);
                    }
                    if (ok && pos < n) {
                        float a, b;
                        f2_split(f2_add(acc[0], acc[1]), a, b);
                        const bool there = good >> (2 * (j - batch) + (me >> 6)) & 1u;
                        float sum = there ? a + b : 0.f;
                        if (p.w_prev && pos < n - w.q.m)
                            sum = fmaf(p.decay, old, sum);
                        p.w[at + pos] = sum;
                    }
                }
            }
            next_unit(w);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

int row_tiles_of(int G, int window) { return (G * window + kBlock - 1) / kBlock; }

}  // namespace

size_t prompt_workspace_bytes(int ctas, int R, int Hkv, int G, int window)
{
    return ((size_t)R * Hkv + ctas) * 2 * row_tiles_of(G, window) * kBlock * sizeof(float2);
}

cudaError_t launch_prompt_weights(const CUtensorMap &tmK, const CUtensorMap &tmQ, const PromptParams &p, int ctas,
                                  cudaStream_t stream)
{
    const size_t smem = sizeof(PromptSmem) + 1024;
    static SmemOptIn opt[2];
    cudaError_t e = opt[0].set(prompt_kernel<1>, smem);
    if (e == cudaSuccess)
        e = opt[1].set(prompt_kernel<2>, smem);
    if (e != cudaSuccess)
        return e;
    const int q_tiles = row_tiles_of(p.G, p.window);
    const int stages = kTiles - q_tiles < kMaxStages ? kTiles - q_tiles : kMaxStages;
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
    e = cudaLaunchKernelEx(&cfg, prompt_kernel<1>, tmK, tmQ, p, q_tiles, stages);
    if (e != cudaSuccess)
        return e;
    return cudaLaunchKernelEx(&cfg, prompt_kernel<2>, tmK, tmQ, p, q_tiles, stages);
}

}  // namespace hsa
