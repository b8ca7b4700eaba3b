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
// owns a key, and the sum over a tile's rows is its own.  Neither sums across threads.  The lse
// goes in through the product: 16 more columns, three ones a key against the three bf16 parts of a
// row's -lse.  (Read from shared memory, 16 bytes to a warp for every four columns, beside the
// products' own reads there, pass 2 took 5% longer.)
//
// Both: persistent, one CTA an SM; the 128-key tiles (two pages) of all (request, KV head) units
// laid end to end and cut into equal ranges.  Warp 0 loads Q (up to four tiles of 128 rows) at a
// unit's start and streams K; warps 1 and 2 issue the MMAs into four TMEM slots of 128 columns, one
// a warpgroup; the four warpgroups of warps 4-19 take the (key tile, row tile) pairs in turn, a
// unit's row tiles (1, 2 or 4 of them in the count: three as four) always the same ones.  In pass 2
// the warpgroups of a key tile hand their sums to the first of them through shared memory.
// The states of a unit's CTAs lie side by side, and every order of summation is fixed.
//
// What bounds it: a warpgroup's chain a tile (2500 cycles for 128 columns; the exponentials alone 2048
// where four warpgroups share the pipe) beside the products.  262144 keys x 4 heads x 512 rows: passes
// of 110 and 128 us, tensor pipe 54%, exponentials 56%, issue 63%; reading K once is 40.  8 requests,
// 256 rows: 138 and 140, and 10% more in an endless loop of them, where the power cap takes the clock.
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
constexpr int kAugBytes = kBlock * 16 * 2; // a tile of 16 columns, K-major without swizzle
constexpr int kGroups = 4;                  // warpgroups, and TMEM slots
constexpr int kIssuers = 2;
constexpr int kThreads = 128 + kGroups * 128;
constexpr uint32_t kTmemCols = 512;
constexpr int kCols = 32;                  // columns a thread takes at a time (16: 299 us for 291)
constexpr float kFar = 0x1p60f;            // of a chunk's sum: its maximum has left the running one behind

struct alignas(1024) PromptSmem {
    uint8_t tile[kTiles][kTileBytes];
    alignas(128) uint8_t ones[kAugBytes];           // pass 2: 16 more columns of K: three of 1
    alignas(128) uint8_t aug[kMaxRowTiles][kAugBytes]; // and of Q: a row's -lse in three parts
    float sum[kGroups][2][kBlock];                  // pass 2: a warpgroup's keys' sums, for the first one
    alignas(8) uint64_t q_full, q_empty, aug_full, done;
    uint64_t k_full[kMaxStages], k_empty[kMaxStages];
    uint64_t s_full[kGroups], s_empty[kGroups];
    uint64_t sum_full[kGroups][2], sum_free[kGroups][2];
    int32_t scan[kThreads];
    int32_t first_r, before, total;
    uint32_t tmem_base;
};

// First byte of a row's columns 0-7 in a tile of 16: groups of eight rows of 16 bytes, the columns
// 8-15 (another such group, always zero here) 128 bytes behind.
__device__ __forceinline__ int aug_offset(int row) { return row / 8 * 256 + row % 8 * 16; }

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

// The block table's entry of page `page` (any value where there is none: page_at tells).  Not looked
// at before it is used: a batch of entries is read while the batch before is on its way.
__device__ __forceinline__ int page_entry(const PromptParams &p, const Request &q, int page)
{
    int blk = 0;
    if ((int64_t)page * 64 < q.n && page < p.max_blocks)
        asm volatile("ld.global.nc.s32 %0, [%1];"
                     : "=r"(blk)
                     : "l"(p.block_tables + (int64_t)q.seq * p.max_blocks + page));
    return blk;
}

// 1: entry blk of page `page` can be read; 0: the page is past the tokens (masked by position); -1:
// out of reach, with *err set.
__device__ __forceinline__ int page_at(const PromptParams &p, const Request &q, int page, int blk, int *err)
{
    if ((int64_t)page * 64 >= q.n)
        return 0;
    if (page < p.max_blocks && blk >= 0 && blk < p.num_blocks)
        return 1;
    *err = page < p.max_blocks ? HSA_DEVERR_BAD_BLOCK : HSA_DEVERR_BAD_PAGE;
    return -1;
}

// Four consecutive 32-bit TMEM columns of this thread's lane (warp-collective).
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
}

// Four sums of 2^(x scale - base) over kCols columns (sc2: the scale twice).
__device__ __forceinline__ void exp_sums(const uint32_t (&x)[kCols], uint64_t sc2, float base, float (&sum)[4])
{
    const uint64_t nb2 = f2_make(-base, -base);
    sum[0] = sum[1] = sum[2] = sum[3] = 0.f;
#pragma unroll
    for (int c = 0; c < kCols; c += 2) {
        float a, b;
        f2_split(f2_fma(f2_make(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, nb2), a, b);
        sum[c & 2] += fast_exp2(a);
        sum[(c & 2) + 1] += fast_exp2(b);
    }
}

// A wait of a whole warp, whose lanes go on together also where it gave up.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity)
{
    return __all_sync(0xffffffffu, mbar_wait_sleep(bar, parity));
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
    if (PASS == 1) {  // (pass 2 waits for it where it needs its sums: the requests are none of its work)
        grid_dependency_wait();
        grid_launch_dependents();
    }

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
    if ((int64_t)blockIdx.x >= C) {
        if (PASS == 2)
            grid_dependency_wait();  // no end of this grid before pass 1's
        return;
    }
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
        mbar_init(&sh.q_empty, kIssuers);
        mbar_init(&sh.done, kIssuers);
        mbar_init(&sh.aug_full, kGroups * kBlock / 32);
        for (int s = 0; s < kMaxStages; ++s) {
            mbar_init(&sh.k_full[s], 1);
            mbar_init(&sh.k_empty[s], kIssuers);
        }
        for (int s = 0; s < kGroups; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.s_empty[s], kBlock / 32);
            for (int e = 0; e < 2; ++e) {
                mbar_init(&sh.sum_full[s][e], kBlock / 32);
                mbar_init(&sh.sum_free[s][e], kBlock / 32);
            }
        }
        fence_barrier_init();
    }
    if (PASS == 2 && tid < kBlock) {
        uint4 *const row = reinterpret_cast<uint4 *>(sh.ones + aug_offset(tid));
        row[0] = make_uint4(0x3f803f80u, 0x3f80u, 0, 0);
        row[8] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    if (PASS == 2)
        grid_dependency_wait();

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
    // pairs are counted tiles x step + row tile, pair e going to warpgroup e mod 4
    auto step_of = [](int nq) { return nq == 3 ? 4 : nq; };

    if (warp == 0) {
        // ------------------------------------------------------------------------ producer
        const uint64_t pol = policy_evict_first();
        int st = 0;          // next stage, and the parity of its phase
        uint32_t ph = 0;
        int issued = 0, units = 0;
        bool ok = true;
        for (int64_t i = kWithholdLoads ? i1 : i0; i < i1 && ok; ++units) {
            const int64_t end = i + min((int64_t)(w.nt - w.j), i1 - i);
            const int nq = row_tiles(w);
            if (units > 0 && !(ok = warp_wait(&sh.q_empty, (uint32_t)(units - 1) & 1)))
                break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sh.q_full, nq * kTileBytes);
                for (int t = 0; t < nq; ++t) {
                    const int row = w.q.row0 + t * (kBlock / p.G);
                    tma_load_3d(sh.tile[t], &tmQ, &sh.q_full, 0, w.h * p.G, row, pol);
                    tma_load_3d(sh.tile[t] + kHalfBytes, &tmQ, &sh.q_full, 64, w.h * p.G, row, pol);
                }
            }
            __syncwarp();
            // pool rows of 32 pages (16 tiles) at a time, a lane each, a batch ahead
            int j = w.j, batch = w.j;
            int cur = page_entry(p, w.q, 2 * batch + lane);
            int nxt = page_entry(p, w.q, 2 * batch + 32 + lane);
            // the pool row of a page, or -1; flagged once, by the first pass
            auto pool_row = [&](int page, int blk) -> int64_t {
                int err = 0;
                if (page_at(p, w.q, page, blk, &err) > 0)
                    return ((int64_t)blk * p.Hkv + w.h) * 64;
                if (PASS == 1 && err && lane == 0)
                    set_err(p.dev_err, err);
                return -1;
            };
            for (; i < end; ++i, ++j) {
                if (j - batch == 16) {
                    batch = j;
                    cur = nxt;
                    nxt = page_entry(p, w.q, 2 * batch + 32 + lane);
                }
                const int b0 = __shfl_sync(0xffffffffu, cur, 2 * (j - batch));
                const int b1 = __shfl_sync(0xffffffffu, cur, 2 * (j - batch) + 1);
                const int64_t y0 = pool_row(2 * j, b0), y1 = pool_row(2 * j + 1, b1);
                const int pages = (y0 >= 0) + (y1 >= 0);
                if (!(ok = warp_wait(&sh.k_empty[st], ph ^ 1)))
                    break;
                uint8_t *dst = sh.tile[q_tiles + st];
                if (elect_one()) {
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
                __syncwarp();
                issued = min(issued + 1, stages);
                if (++st == stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            next_unit(w);
        }
        if (lane == 0) {
            if (!ok)
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
            // no copy may still be in flight when the CTA exits
            for (int s = 0; s < issued; ++s)
                mbar_wait_sleep(&sh.k_full[s], s < st ? ph : ph ^ 1);
            if (units > 0)
                mbar_wait_sleep(&sh.q_full, (uint32_t)(units - 1) & 1);
        }
    } else if (warp <= kIssuers) {
        // --------------------------------------------------------------------- MMA issuers
        // Issuer u serves the warpgroups u and u + 2.  The whole warp runs the loop and one
        // elected lane issues: control flow and descriptors stay uniform.
        const int u = warp - 1;
        const uint32_t dhi = smem_desc_sw128_hi(1024);
        auto commit = [&](uint64_t *bar) {
            if (elect_one())
                tc_commit(bar);
        };
        // a tile of 16 columns: no swizzle, 128 bytes from its columns 0-7 to 8-15, 256 from eight
        // rows to the next
        auto aug_desc = [](const uint8_t *tile) -> uint64_t {
            return (uint64_t)(smem_u32(tile) >> 4) | (uint64_t)(128 >> 4) << 16 | (uint64_t)(256 >> 4) << 32 | 1ull << 46;
        };
        int st = 0, units = 0;
        uint32_t ph = 0;
        uint32_t given = 0;  // bit wg: parity of the tiles handed to warpgroup wg
        bool ok = true;
        for (int64_t i = i0; i < i1 && ok; ++units) {
            const int tiles = (int)min((int64_t)(w.nt - w.j), i1 - i);
            const int nq = row_tiles(w), rows = w.q.T * p.G, step = step_of(nq);
            ok = warp_wait(&sh.q_full, (uint32_t)units & 1) &&
                 (PASS == 1 || warp_wait(&sh.aug_full, (uint32_t)units & 1));
            for (int e = 0; e < tiles && ok; ++e) {
                if (!(ok = warp_wait(&sh.k_full[st], ph)))
                    break;
                tc_fence_after();
                const uint32_t kl = smem_desc_sw128_lo(smem_u32(sh.tile[q_tiles + st]), 16);
                for (int t = 0; t < nq; ++t) {
                    const int slot = (e * step + t) & (kGroups - 1);
                    if ((slot & 1) != u)
                        continue;
                    if (!(ok = warp_wait(&sh.s_empty[slot], (given >> slot & 1) ^ 1)))
                        break;
                    given ^= 1u << slot;
                    tc_fence_after();
                    const uint32_t ql = smem_desc_sw128_lo(smem_u32(sh.tile[t]), 16);
                    const int cols = PASS == 1 ? kBlock : min(kBlock, (rows - t * kBlock + 15) & ~15);
                    const uint32_t id = idesc_bf16_f32(kBlock, cols, 0, 0);
                    const uint32_t a = PASS == 1 ? ql : kl, b = PASS == 1 ? kl : ql;
                    const uint32_t d = tmem + slot * kBlock;
                    const bool one = elect_one();
#pragma unroll
                    for (int ks = 0; ks < kD / 16; ++ks) {
                        const uint32_t off = (ks >> 2) * (kHalfBytes >> 4) + (ks & 3) * 2;
                        if (one) {
                            if (ks == 0)
                                tc_mma_ss_k<0>(d, desc_join(a, dhi), desc_join(b, dhi), id);
                            else
                                tc_mma_ss_k<1>(d, desc_join(a + off, dhi), desc_join(b + off, dhi), id);
                        }
                    }
                    if (PASS == 2 && one)  // S^T - lse
                        tc_mma_ss_k<1>(d, aug_desc(sh.ones), aug_desc(sh.aug[t]), id);
                    commit(&sh.s_full[slot]);
                }
                if (!ok)
                    break;
                commit(&sh.k_empty[st]);  // arrives at once where nothing was issued
                if (++st == stages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if (ok)
                commit(&sh.q_empty);
            i += tiles;
            next_unit(w);
        }
        if (!ok && lane == 0)
            set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
        commit(&sh.done);  // every MMA done before TMEM is released
        mbar_wait_sleep(&sh.done, 0);
    } else if (warp >= 4) {
        // ------------------------------------------------------------- rows' or keys' threads
        const int wg = (warp - 4) >> 2, wq = warp & 3;
        const int me = wq * 32 + lane;  // TMEM lane
        const uint32_t taddr = tmem + ((uint32_t)(wq * 32) << 16) + wg * kBlock;
        const uint64_t sc2 = f2_make(p.scale_log2, p.scale_log2);
        uint32_t cnt = 0;       // tiles taken
        int units = 0;
        uint32_t handed = 0;    // pass 2: byte g: sums that warpgroup g has handed over, mod 4
        bool ok = true;
        // bit e: page 2 batch + e can be read
        auto pages_ok = [&](int batch) {
            const int page = 2 * batch + lane;
            int err;
            return __ballot_sync(0xffffffffu, page_at(p, w.q, page, page_entry(p, w.q, page), &err) >= 0);
        };
        // After a wait that gave up no further one is made, but every tile is walked through: the
        // warpgroup's barriers count on all of it.
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            if (ok && !mbar_wait_sleep(bar, parity)) {
                set_err(p.dev_err, HSA_DEVERR_TIMEOUT);
                ok = false;
            }
            __syncwarp();
        };
        auto take = [&] {
            wait(&sh.s_full[wg], cnt & 1);
            tc_fence_after();
        };
        auto arrive = [&](uint64_t *bar) {  // a warp's one
            __syncwarp();
            if (lane == 0)
                mbar_arrive(bar);
        };
        auto give = [&] {
            tc_fence_before();
            arrive(&sh.s_empty[wg]);
            ++cnt;
        };
        for (int64_t i = i0; i < i1;) {
            const int64_t unit = (int64_t)w.r * p.Hkv + w.h;
            const int tiles = (int)min((int64_t)(w.nt - w.j), i1 - i);
            const int nq = row_tiles(w), step = step_of(nq), n = w.q.n, T = w.q.T, rows = T * p.G;
            const int t = wg % step;  // this warpgroup's row tile
            const int row0 = t * kBlock;
            int batch = w.j;
            uint32_t good = pages_ok(batch);
            if constexpr (PASS == 1) {
                // the sum with what its roundings lost (a row has up to a million terms)
                float m = -INFINITY, l = 0.f, lost = 0.f;
                const int sees = min(n, n - T + (row0 + me) / p.G + 1);  // keys that this row sees
                for (int e = wg / step; t < nq && e < tiles; e += kGroups / step) {
                    const int j = w.j + e;
                    if (j - batch >= 16) {
                        batch += (j - batch) & ~15;
                        good = pages_ok(batch);
                    }
                    const uint32_t pair = good >> (2 * (j - batch)) & 3u;
                    // keys of the tile this row sees: 0 .. hi - 1
                    const int hi = sees - j * kBlock;
                    const bool whole = __all_sync(0xffffffffu, hi >= kBlock) && pair == 3u;
                    take();
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
                    for (int c0 = 0; c0 < kBlock; c0 += kCols) {
                        uint32_t x[kCols];
                        tmem_ld32(taddr + c0, x);
                        tmem_wait_ld();
                        if (c0 == kBlock - kCols)
                            give();
                        if (!whole) {
                            const int top = (pair >> (c0 >> 6) & 1u) ? hi - c0 : 0;
#pragma unroll
                            for (int c = 0; c < kCols; ++c)
                                if (c >= top)
                                    x[c] = __float_as_uint(-INFINITY);
                        }
                        // the exponents take the maximum as of the chunks before.  A sum that
                        // leaves fp32's middle says that this chunk's is far above it; only
                        // then, and at the first, is it sought.
                        float part[4];
                        const float base = m == -INFINITY ? 0.f : m;
                        exp_sums(x, sc2, base, part);
                        const float all = (part[0] + part[1]) + (part[2] + part[3]);
                        if (m == -INFINITY || !(all < kFar)) {
                            float top = -INFINITY;
#pragma unroll
                            for (int c = 0; c < kCols; c += 2)
                                top = fmax3(top, __uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                            top *= p.scale_log2;
                            if (top != -INFINITY && (m == -INFINITY || top > m)) {
                                const float f = m == -INFINITY ? 0.f : fast_exp2(m - top);
                                l *= f;
                                lost *= f;
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    acc[c] *= f;
                                m = top;
                                exp_sums(x, sc2, top, part);
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            acc[c] += part[c];
                    }
                    const float add = ((acc[0] + acc[1]) + (acc[2] + acc[3])) - lost, sum = l + add;
                    lost = (sum - l) - add;
                    l = sum;
                }
                p.part[((unit + blockIdx.x) * kGroups + wg) * kBlock + me] = make_float2(m, l);
            } else {
                // ---- the rows' lse, out of the states of every CTA that met the unit: those of
                // the warpgroups t, t + step, .. of each
                {
                    const int64_t u0 = i - w.j, u1 = u0 + w.nt;
                    const int64_t c_lo = ((u0 + 1) * C - 1) / N, c_hi = (u1 * C - 1) / N;
                    const float2 *const part = p.part + (unit + c_lo) * kGroups * kBlock + me;
                    const int states = (int)(c_hi - c_lo + 1) * kGroups;
                    float M = -INFINITY, L = 0.f;
                    for (int e0 = t; e0 < states; e0 += 8 * step) {
                        float2 s[8];
                        float top = M;
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            s[e] = make_float2(-INFINITY, 0.f);
                            if (e0 + e * step < states)
                                s[e] = __ldcg(part + (int64_t)(e0 + e * step) * kBlock);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            top = fmaxf(top, s[e].x);
                        const float base = top == -INFINITY ? 0.f : top;
                        L *= fast_exp2(M - base);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            L += s[e].y * fast_exp2(s[e].x - base);
                        M = top;
                    }
                    // -lse in units of a raw score, as a sum of three bf16; where there is no row, or
                    // no key, what leaves no weight.  (NaN passes.)
                    const bool on = row0 + me < rows && L != 0.f;
                    const float v = on ? -((M == -INFINITY ? 0.f : M) + log2f(L)) / p.scale_log2 : -1e30f;
                    const uint32_t hi = pack_bf16(v, 0.f) & 0xffffu;
                    const float rest = on ? v - bf16_lo(hi) : 0.f;
                    const uint32_t mid = pack_bf16(rest, 0.f) & 0xffffu;
                    const uint32_t lo = pack_bf16(on ? rest - bf16_lo(mid) : 0.f, 0.f) & 0xffffu;
                    if (units > 0)
                        wait(&sh.q_empty, (uint32_t)(units - 1) & 1);  // the last unit's products are done
                    if (wg < step) {
                        uint4 *const row = reinterpret_cast<uint4 *>(sh.aug[t] + aug_offset(me));
                        row[0] = make_uint4(hi | mid << 16, lo, 0, 0);
                        row[8] = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    arrive(&sh.aug_full);
                }
                const int64_t at = ((int64_t)w.q.seq * p.Hkv + w.h) * p.w_stride;
                const int top = min(kBlock, rows - row0);
                uint32_t turn = 0;  // key tiles of this warpgroup (and of those it shares them with)
                for (int e = wg / step; t < nq && e < tiles; e += kGroups / step, ++turn) {
                    const int j = w.j + e;
                    if (j - batch >= 16) {
                        batch += (j - batch) & ~15;
                        good = pages_ok(batch);
                    }
                    const int pos = j * kBlock + me;
                    const int first = max(0, pos - (n - T)) * p.G - row0;  // of the tile's rows, first .. see the key
                    const bool all = __all_sync(0xffffffffu, first <= 0);
                    const float old = t == 0 && p.w_prev && pos < n - w.q.m ? p.w_prev[at + pos] : 0.f;
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
                    take();
                    if (all && top == kBlock) {
#pragma unroll 1
                        for (int c0 = 0; c0 < kBlock; c0 += kCols) {
                            uint32_t x[kCols];
                            tmem_ld32(taddr + c0, x);
                            tmem_wait_ld();
                            if (c0 == kBlock - kCols)
                                give();
#pragma unroll
                            for (int c = 0; c < kCols; c += 2) {
                                float a, b;
                                f2_split(f2_mul(f2_make(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2), a, b);
                                acc[c & 2] += fast_exp2(a);
                                acc[(c & 2) + 1] += fast_exp2(b);
                            }
                        }
                    } else {
                        // rows that do not see the key, or that there are not
#pragma unroll 1
                        for (int c0 = 0; c0 < top; c0 += 4) {
                            uint32_t x[4];
                            tmem_ld4(taddr + c0, x);
                            tmem_wait_ld();
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c0 + c >= first && c0 + c < top)
                                    acc[c] += fast_exp2(__uint_as_float(x[c]) * p.scale_log2);
                        }
                        give();
                    }
                    float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
                    if (t > 0) {  // over to the key tile's first warpgroup
                        const uint32_t c = (handed >> (8 * wg)) + turn;
                        wait(&sh.sum_free[wg][c & 1], (c >> 1 & 1) ^ 1);
                        sh.sum[wg][c & 1][me] = sum;
                        arrive(&sh.sum_full[wg][c & 1]);
                        continue;
                    }
                    for (int g = wg + 1; g < wg + nq; ++g) {
                        const uint32_t c = (handed >> (8 * g)) + turn;
                        wait(&sh.sum_full[g][c & 1], c >> 1 & 1);
                        sum += sh.sum[g][c & 1][me];
                        arrive(&sh.sum_free[g][c & 1]);
                    }
                    if (ok && pos < n) {
                        sum = good >> (2 * (j - batch) + (me >> 6)) & 1u ? sum : 0.f;
                        if (p.w_prev && pos < n - w.q.m)
                            sum = fmaf(p.decay, old, sum);
                        p.w[at + pos] = sum;
                    }
                }
                for (int g = 0; g < kGroups; ++g)
                    if (g % step > 0 && g % step < nq)
                        handed += (uint32_t)max(0, (tiles - g / step + kGroups / step - 1) / (kGroups / step)) % 4 << (8 * g);
                handed &= 0x03030303u;
            }
            i += tiles;
            ++units;
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

size_t prompt_workspace_bytes(int ctas, int R, int Hkv)
{
    return ((size_t)R * Hkv + ctas) * kGroups * kBlock * sizeof(float2);
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
