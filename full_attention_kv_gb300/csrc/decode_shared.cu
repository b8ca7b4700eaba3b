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
// attend_kernel, part 1 (tcgen05): the query rows of a group for one KV head -- members x T
// tokens x G heads -- are packed into 128-row tiles, a pair of tiles (256 rows) a unit, and
// meet the shared keys page by page as a dense product: K and V are read once a unit
// instead of once a sequence.  The pages of all units are laid end to end and cut into
// equal ranges, one per CTA; each (CTA, unit) segment leaves unnormalised fp32 states.
// Part 2 (mma.sync, 8 to 32 rows a sequence and head): a stream-K walk over the pages past
// the shared ones and the new tokens; each segment leaves its state.  The parts were two
// kernels first; between them an SM stood idle for about 9 us (part 1's states, 133 KB a CTA,
// drain before a CTA's place is free, then part 2's launch and plan).  In one kernel part 2's
// plan is made by a spare warp during part 1, and its first loads pass the draining states.
// merge_kernel: merges each row's states and writes bf16; it also appends the new rows.
//
// What bounds it (152 SMs; measured peaks 6.8 TB/s and 1.94 PFLOP/s; whole calls): many rows a
// page, the tensor cores (128 sequences on a document of 65600 tokens, 32 / 4 heads, 130 us:
// 1.07 PFLOP/s); few rows a page, the reads (32 sequences in 12 groups of 1 to 5 on prompts of
// 1000 to 40000 tokens, 88 us: 5.5 TB/s); between them the two parts one after the other and
// their seams (32 sequences on 32768 tokens with 64 to 4096 of their own, 56 us: 3.6 TB/s); four
// samples of one prompt of 2048 tokens, latency (15 us).  decode.cu takes 1750, 234, 279 and
// 224 us for the four; the last is its merge, which takes a unit's states one after the other
// (8 units over 152 CTAs; 39 us over 16).
// Part 2 beside part 1 instead of after it (warps of its own, registers shared out by
// setmaxnreg) measured 141 us for the document and 87 against 80 for 48 verified drafts: its
// mma.sync products share the tensor cores, and it has half of the stages.
// Items and parts are counted in 32 bits: 64-bit divisions and the registers they held cost
// the document 11 us and the four samples 4.
#include "decode_tile.cuh"
#include "hsa_device.cuh"
#include "hsa_internal.h"

namespace hsa {
namespace {

// ------------------------------------------------------------------ groups

__device__ __forceinline__ int clamp_len(int c) { return c < 0 ? 0 : c; }

// A group's shared whole pages, or 0 (nothing is shared): as many as the first member, whose
// row they are read through, has cached.  Behind its own tokens a row may hold anything, and
// so may a page that nobody has written; a later member's further pages are its own.
// (Offsets in order.)
__device__ __forceinline__ int group_pages(const SharedParams &p, int g)
{
    const int b = __ldg(p.cu_group + g);
    if (b >= __ldg(p.cu_group + g + 1))
        return 0;
    const int len = min(__ldg(p.shared_len + g), __ldg(p.d.cached_len + b));
    return min(clamp_len(len) / kTileKeys, p.d.max_blocks);
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

// ------------------------------------------------------------------ part 1: shared pages
//
// A step is one 64-key page.  Each query tile has two 64-column S regions in TMEM, so that
// the next page's scores are there when the softmax warps finish a page.
//   pair mode (129 .. 256 rows): query tiles A and B, one warpgroup each, every page
//   split mode (up to 128 rows): one query tile; the warpgroups, with S and O regions of
//     their own, take the pages in turn and leave two states a row
// Each warpgroup has an issuing warp of its own: one warp issues a product in about 90 cycles
// and spends a third of a step in the latency of its waits and commits, and two of them keep
// the tensor cores fed (one for both tiles, S of one between PV of the other: 186 us against
// 131 for the document; a third for PV: 135).  A step of
// a pair takes about 1550 cycles.  Its products take about 1440: 64 cycles for a k-step of PV,
// and 58 for one of S, whose arithmetic takes 32 but which reads 6 KB of shared memory.  (S of
// two pages at a time reads less, but leaves TMEM one region a tile and the softmax waiting:
// 131 us against 109 for part 1 of the document.)  The softmax warps take about 1180.
// K and V pages pass through a ring of two-page stages in the order of their use: with L = 2
// (pair) or 4 (split) pages of scores ahead, [K0 K1] .. [K(L-2) K(L-1)], then [V(n) K(n+L)].

constexpr int kBM = 128;
constexpr int kQBytes = kBM * kD * 2;       // 32 KB: two blocks of 128 rows x 64 columns
constexpr int kQHalf = kQBytes / 2;
constexpr int kPageBytes = kTileKeys * kD * 2;  // 16 KB: two blocks of 64 rows x 64 columns
constexpr int kPageHalf = kPageBytes / 2;
constexpr int kRing = 5;
constexpr int kAttendThreads = 384;         // producer 0, issuers 1 and 10, softmax 2 .. 9, plan 11
// Log2 units that P may lie above 1 before O is rescaled at once: more than usual pages rise,
// and few enough that O has room for values up to 2^127 / 2^16 less the keys' count.
constexpr float kFar = 16.0f;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;             // S: tile t, region h at 128 t + 64 h; O_t at 256 + 128 t
// A segment's states, by octets of rows: m[8], l[8], then o as [dim / 4][8 rows][4], so
// that the warps that write (a row a lane) and those that merge (eight rows x four
// 16-byte pieces) both move whole 128-byte lines.
constexpr int kOctFloats = 16 + 8 * kD;
constexpr int kSlotFloats = 2 * kBM / 8 * kOctFloats;

// First item of part c <= C of N items cut into C equal parts: floor(c N / C).  (shared_fits
// bounds N, and C < 2^16.)
__device__ __forceinline__ int cut(int c, int N, int C)
{
    const uint32_t q = (uint32_t)N / (uint32_t)C;
    return (int)(c * q + c * ((uint32_t)N - q * C) / (uint32_t)C);
}

// The part that holds item s: the c with cut(c) <= s < cut(c + 1), from a guess that is off by
// one at most.
__device__ __forceinline__ int part_of(int s, int N, int C)
{
    int c = min((int)((float)s * ((float)C / (float)N)), C - 1);
    if (cut(c, N, C) > s)
        --c;
    else if (cut(c + 1, N, C) <= s)
        ++c;
    return c;
}

// A page of a unit in pair mode counts two items, one of a unit in split mode (a group's
// last 128 rows or fewer) one: with equal items the CTAs that drew split units were done
// after 31 us and the others after 57 (three groups of 96, 352 and 1088 rows).  A page belongs
// to the CTA that holds its first item.
__host__ __device__ inline int page_items(int rows) { return rows <= kBM ? 1 : 2; }

// A group's items for one head: units of 256 rows, the last one's weight by its rows.
__host__ __device__ inline int head_items(int pairs, int pages, int rows)
{
    return pairs > 0 ? pages * (2 * (pairs - 1) + page_items(rows - (pairs - 1) * 2 * kBM)) : 0;
}

// Parts that N items are cut into: of two items at least, so that every part of a unit
// between its first page's and its last page's holds a page.
__host__ __device__ inline int item_parts(int N, int ctas)
{
    return N < 2 * ctas ? (N + 1) / 2 : ctas;
}

// A CTA's walk over the segments of its item range: every role runs its own copy.
struct SegWalk {
    int it, i1, item0;  // next item, end, first item of group g
    int per_head;       // the group's items a head
    int g, unit0;       // group, units before it
    int pairs, pages;   // the group's 256-row units a head, pages a unit
    int seq0, ntok;
    // the current segment: pages n0 .. n1 - 1
    int h, pair, n0, n1, unit, rows;
    __device__ __forceinline__ bool split() const { return rows <= kBM; }
};

__device__ __forceinline__ void load_group(const SharedParams &p, SegWalk &w)
{
    w.seq0 = __ldg(p.cu_group + w.g);
    w.ntok = (__ldg(p.cu_group + w.g + 1) - w.seq0) * p.d.T;
    w.pages = group_pages(p, w.g);
    w.pairs = w.pages > 0 ? (w.ntok * p.d.G + 2 * kBM - 1) / (2 * kBM) : 0;
    w.per_head = head_items(w.pairs, w.pages, w.ntok * p.d.G);
}

__device__ __forceinline__ bool next_seg(const SharedParams &p, SegWalk &w)
{
    while (w.it < w.i1) {
        while (w.it >= w.item0 + w.per_head * p.d.Hkv) {
            w.item0 += w.per_head * p.d.Hkv;
            w.unit0 += w.pairs * p.d.Hkv;
            ++w.g;
            load_group(p, w);
        }
        const uint32_t off = w.it - w.item0;
        w.h = (int)(off / (uint32_t)w.per_head);
        const int in_head = (int)(off - w.h * w.per_head);
        w.pair = min((int)((uint32_t)in_head / (2u * w.pages)), w.pairs - 1);
        w.unit = w.unit0 + w.h * w.pairs + w.pair;
        w.rows = w.ntok * p.d.G - w.pair * 2 * kBM;
        const int wt = page_items(w.rows);
        const int o0 = in_head - w.pair * 2 * w.pages;  // items into the unit
        const int o1 = min(w.pages * wt, o0 + (w.i1 - w.it));
        w.it += o1 - o0;
        w.n0 = (o0 + wt - 1) >> (wt - 1);  // wt is 1 or 2
        w.n1 = (o1 + wt - 1) >> (wt - 1);
        if (w.n0 < w.n1)
            return true;
    }
    return false;
}

__device__ __forceinline__ bool page_ok(const SharedParams &p, int seq, int page, int *blk)
{
    const int b = __ldg(p.d.block_tables + (int64_t)seq * p.d.max_blocks + page);
    if (b < 0 || b >= p.d.num_blocks)
        return false;
    *blk = b;
    return true;
}

// ------------------------------------------------------ part 2: own pages and new tokens
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
// A unit counts kUnitCost items more than it has keys for: starting and leaving one (query
// rows, new rows, state) takes a group about as long, and without it the streams that cross
// many short units ended last (a batch of 1 .. 1024 own tokens: 28 us the median stream, 46
// the last).  Those items, the unit's first, do nothing.
constexpr int kUnitCost = 2;
constexpr int kInfoCap = 128;                   // sequences whose lengths are kept in shared memory

struct OwnSmem {
    alignas(8) uint64_t full[kGroups][kDepth];
    alignas(8) uint64_t empty[kGroups][kDepth];  // MT = 2: the second warp is done with it
    int32_t ok[kGroups][kDepth];                 // the item's cached keys were loaded
    int2 info[kInfoCap];                         // (c, fp) of a sequence
    int32_t first_b[kGroups], first_before[kGroups];
    int32_t total_items, share;
    alignas(8) uint64_t ready;                   // the plan is made
};

// Position in a stream: sequence b, head h, item j of n; c cached tokens past the first
// page `fp` that is the sequence's own.
struct OwnWalk {
    int b, h, j, n, c, fp;
    __device__ __forceinline__ int key0() const { return (j - kUnitCost) * kKT; }  // < 0: no keys
};

// c and fp of sequence b, from the inputs.
__device__ __forceinline__ int2 own_info(const SharedParams &p, bool share, int b)
{
    const int fp = share ? group_pages(p, group_of(p, b)) : 0;
    // a length past the block table counts up to the first page that is not there
    const int64_t most = ((int64_t)p.d.max_blocks + 1) * kTileKeys;
    const int c = (int)min((int64_t)clamp_len(__ldg(p.d.cached_len + b)), most);
    return make_int2(max(0, c - fp * kTileKeys), fp);
}

__device__ __forceinline__ int own_items(const SharedParams &p, int c)
{
    return kUnitCost + (c + p.d.T + kKT - 1) / kKT;
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
    const int k0 = w.key0(), page = w.fp + k0 / kTileKeys;
    if (k0 < 0 || k0 >= w.c || page >= p.d.max_blocks)
        return -1;
    return __ldg(p.d.block_tables + (int64_t)w.b * p.d.max_blocks + page);
}

// Floats of an own segment's state: m[R], l[R], o[R][128] for R = G T rows, m and l padded
// to 16 bytes.
__host__ __device__ inline int own_pad(int rows) { return (rows + 3) & ~3; }
__host__ __device__ inline int own_slot_floats(int rows) { return 2 * own_pad(rows) + rows * kD; }

// The stream of this CTA's group grp.  Streams 0 .. gridDim - 1 are on different CTAs, so that
// few items still use every SM, and the first on the last CTA: where part 1 has fewer parts
// than there are CTAs, the two parts' work is on different ones.
__device__ __forceinline__ int own_stream(int grp)
{
    return grp * (int)gridDim.x + ((int)gridDim.x - 1 - (int)blockIdx.x);
}

// Part 2's plan, by one warp: the items before each sequence, and where this CTA's streams
// begin.
__device__ __forceinline__ void own_plan(const SharedParams &p, OwnSmem &sh, int lane)
{
    const DecodeParams &d = p.d;
    const bool share = groups_ok(p, lane);
    OwnPlan *const plan = reinterpret_cast<OwnPlan *>(d.ws + p.own_plan_off);
    int total = 0;
    for (int base = 0; base < d.B; base += 32) {
        const int b = base + lane;
        int n = 0;
        if (b < d.B) {
            const int2 v = own_info(p, share, b);
            if (b < kInfoCap)
                sh.info[b] = v;
            n = own_items(p, v.x);
        }
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        if (blockIdx.x == 0 && b < d.B)  // for the merge
            plan->before[b] = total + incl - n;
        total += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int N = total * d.Hkv, C = min(N, (int)gridDim.x * kGroups);
    if (lane == 0) {
        sh.share = share;
        sh.total_items = total;
        if (blockIdx.x == 0) {
            plan->N = N;
            plan->C = C;
        }
    }
    // second walk: the sequences that hold the first items of this CTA's streams
    int at[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i)
        at[i] = own_stream(i) < C ? cut(own_stream(i), N, C) : N;
    __syncwarp();
    int before = 0;
    for (int base = 0; base < d.B; base += 32) {
        const int b = base + lane;
        int n = 0;
        if (b < d.B)
            n = own_items(p, b < kInfoCap ? sh.info[b].x : own_info(p, share, b).x);
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += u;
        }
        const int lo = before + incl - n;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
            if (n > 0 && lo * d.Hkv <= at[i] && (lo + n) * d.Hkv > at[i]) {
                sh.first_b[i] = b;
                sh.first_before[i] = lo;
            }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
}

// The position of a stream's first item.
__device__ __forceinline__ OwnWalk own_start(const SharedParams &p, const OwnSmem &sh, int grp,
                                             int i0)
{
    OwnWalk w;
    w.b = sh.first_b[grp];
    own_load(p, sh, w);
    const int off = i0 - sh.first_before[grp] * p.d.Hkv;
    w.h = off / w.n;
    w.j = off - w.h * w.n;
    return w;
}

// The streams of this CTA: group grp, warp mt of its MT.
template <int MT>
__device__ __forceinline__ void own_run(const CUtensorMap &tmK, const CUtensorMap &tmV,
                                        const SharedParams &p, OwnSmem &sh,
                                        uint8_t (*stages)[kDepth][kItemBytes], int grp, int mt,
                                        int lane)
{
    const DecodeParams &d = p.d;
    const int N = sh.total_items * d.Hkv, C = min(N, (int)gridDim.x * kGroups);
    const int stream = own_stream(grp);
    if (stream >= C)
        return;
    const int i0 = cut(stream, N, C), i1 = cut(stream + 1, N, C);
    OwnWalk w = own_start(p, sh, grp, i0);

    // ---- loads: item li of the stream, kDepth items ahead of the products ------------
    const uint64_t pol = policy_evict_first();
    OwnWalk lw = w;
    int li = i0;
    int lst = 0;
    uint32_t lph = 0;  // parity of the stage's next empty phase (MT = 2)
    auto skip = [&] {  // to an item with keys
        while (li < i1 && lw.key0() < 0) {
            ++li;
            if (li < i1)
                own_next(p, sh, lw);
        }
    };
    skip();
    int entry = li < i1 ? own_entry(p, lw) : -1;
    auto load = [&](bool refill) {  // the group's first warp
        if (li >= i1)
            return;
        if (MT == 2 && refill && !mbar_wait(&sh.empty[grp][lst], lph)) {
            set_err(d.dev_err, HSA_DEVERR_TIMEOUT);
            li = i1;  // no more loads: the products then give up on their own
            return;
        }
        if (lane == 0) {
            const int k0 = lw.key0();
            bool ok = k0 < lw.c;
            if (ok && (entry < 0 || entry >= d.num_blocks)) {
                set_err(d.dev_err, lw.fp + k0 / kTileKeys >= d.max_blocks ? HSA_DEVERR_BAD_PAGE
                                                                         : HSA_DEVERR_BAD_BLOCK);
                ok = false;
            }
            uint64_t *const full = &sh.full[grp][lst];
            sh.ok[grp][lst] = ok;
            if (ok) {
                uint8_t *const dst = stages[grp][lst];
                const int32_t r = (entry * d.Hkv + lw.h) * kTileKeys + k0 % kTileKeys;
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
            skip();
            if (li < i1)
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
    const int pad = own_pad(rows);
    bool fresh = true, timed_out = false;
    for (int i = i0; i < i1; ++i) {
        if (w.key0() < 0) {
            if (i == i1 - 1) {  // the share holds no keys
                float *const part = reinterpret_cast<float *>(d.ws + p.own_off) +
                                    (int64_t)(stream + w.b * d.Hkv + w.h) * own_slot_floats(rows);
                for (int e = lane; e < min(16, rows - mt * 16); e += 32) {
                    part[mt * 16 + e] = -INFINITY;
                    part[pad + mt * 16 + e] = 0.f;
                }
                for (int e = lane; e < min(16, rows - mt * 16) * (kD / 4); e += 32)
                    reinterpret_cast<float4 *>(part + 2 * pad + mt * 16 * kD)[e] =
                        make_float4(0.f, 0.f, 0.f, 0.f);
            }
            own_next(p, sh, w);
            continue;
        }
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
            li = i1;
            for (int s = 0; s < kDepth; ++s)  // no TMA write may be in flight when the CTA exits
                mbar_wait(&sh.full[grp][s], s < stg ? ph ^ 1 : ph);
        }
        uint8_t *const base = stages[grp][stg];
        // keys 0 .. cached - 1 of the item are cached ones, key news + t is new token t
        const int news = w.c - w.key0();
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
            float *const part = reinterpret_cast<float *>(d.ws + p.own_off) +
                                (int64_t)(stream + w.b * d.Hkv + w.h) * own_slot_floats(rows);
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
}

struct AttendSmem {
    // part 2's stages lie over these
    alignas(1024) uint8_t q[2][kQBytes];
    alignas(1024) uint8_t ring[kRing][2][kPageBytes];
    alignas(8) uint64_t q_full, q_empty;
    uint64_t full[kRing], empty[kRing];
    uint64_t s_full[2][2], p_full[2][2];    // [query tile][region]
    uint64_t pv_done[2], o_empty[2], done[2];
    uint32_t tmem_base;
    int32_t g0, unit0, item0, N;
    OwnSmem own;
};
static_assert(kGroups * kDepth * kItemBytes <= 2 * kQBytes + 2 * kRing * kPageBytes, "part 2's stages");
static_assert(sizeof(AttendSmem) + 1024 <= 232448, "shared memory");

// Position in the ring: buffer and the parity of its current phase.
struct RingPos {
    int b;
    uint32_t ph;
    __device__ __forceinline__ void next()
    {
        if (++b == kRing) {
            b = 0;
            ph ^= 1;
        }
    }
};

// MT: 16-row m-tiles of a sequence's G T query rows (1 or 2), a warp each in part 2.
template <int MT>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK32,
                  const __grid_constant__ CUtensorMap tmV32, const __grid_constant__ SharedParams p)
{
    extern __shared__ uint8_t smem_raw[];
    AttendSmem &sh = *reinterpret_cast<AttendSmem *>(align_smem_1024(smem_raw));
    const int tid = threadIdx.x;
    const int warp = tid >> 5, lane = tid & 31;

    if (tid == 32) {
        mbar_init(&sh.q_full, 1);
        mbar_init(&sh.q_empty, 2);  // here and for a stage: the two issuers
        for (int s = 0; s < kRing; ++s) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 2);
        }
        for (int t = 0; t < 2; ++t) {
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sh.s_full[t][h], 1);
                mbar_init(&sh.p_full[t][h], 4);  // its warps
            }
            mbar_init(&sh.pv_done[t], 1);
            mbar_init(&sh.o_empty[t], 4);
            mbar_init(&sh.done[t], 1);
        }
        mbar_init(&sh.own.ready, 1);
        for (int i = 0; i < kGroups; ++i)
            for (int s = 0; s < kDepth; ++s) {
                mbar_init(&sh.own.full[i][s], 1);
                mbar_init(&sh.own.empty[i][s], 1);
            }
        fence_barrier_init();
    }
    if (tid == 64) {
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
        tma_prefetch_desc(&tmK32);
        tma_prefetch_desc(&tmV32);
    }
    if (warp == 1) {
        __syncwarp();
        tmem_alloc(&sh.tmem_base, kTmemCols);
        tmem_relinquish();
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the item space: warp 0 sums the groups and finds this CTA's first item ------
    if (warp == 0) {
        const bool ok = groups_ok(p, lane);
        SharedPlan *const plan = reinterpret_cast<SharedPlan *>(p.d.ws + p.plan_off);
        int N = 0, C = 0, i0 = 0;
        for (int walk = 0; walk < 2; ++walk) {  // 0: the sums, 1: the group that holds i0
            int total = 0, units = 0;
            for (int base = 0; ok && base < p.n_groups; base += 32) {
                SegWalk w{};
                w.g = base + lane;
                if (w.g < p.n_groups)
                    load_group(p, w);
                const int n = w.per_head * p.d.Hkv, un = w.pairs * p.d.Hkv;
                int incl = n, uincl = un;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int a = __shfl_up_sync(0xffffffffu, incl, o);
                    const int b = __shfl_up_sync(0xffffffffu, uincl, o);
                    if (lane >= o) {
                        incl += a;
                        uincl += b;
                    }
                }
                if (walk == 0 && blockIdx.x == 0 && w.g < p.n_groups) {
                    SharedGroup &gp = plan->group[w.g];
                    gp.item0 = total + incl - n;
                    gp.unit0 = units + uincl - un;
                    gp.pairs = w.pairs;
                    gp.pages = w.pages;
                    const int len = __ldg(p.shared_len + w.g);
                    if (len < 0)
                        set_err(p.d.dev_err, HSA_DEVERR_BAD_LEN);
                    if (len / kTileKeys > p.d.max_blocks)
                        set_err(p.d.dev_err, HSA_DEVERR_BAD_PAGE);
                }
                if (walk == 1 && total + incl - n <= i0 && i0 < total + incl) {
                    sh.g0 = w.g;
                    sh.unit0 = units + uincl - un;
                    sh.item0 = total + incl - n;
                }
                total += __shfl_sync(0xffffffffu, incl, 31);
                units += __shfl_sync(0xffffffffu, uincl, 31);
            }
            if (walk == 0) {
                N = total;
                C = item_parts(N, gridDim.x);
                i0 = (int)blockIdx.x < C ? cut(blockIdx.x, N, C) : N;
                if (lane == 0)
                    sh.N = N;
                if (blockIdx.x == 0 && lane == 0) {
                    plan->N = N;
                    plan->C = C;
                    if (!ok)
                        set_err(p.d.dev_err, HSA_DEVERR_BAD_LEN);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int N = sh.N, C = item_parts(N, gridDim.x);
    SegWalk w{};
    if ((int)blockIdx.x < C) {  // else no segments
        w.it = cut(blockIdx.x, N, C);
        w.i1 = cut((int)blockIdx.x + 1, N, C);
        w.item0 = sh.item0;
        w.g = sh.g0;
        w.unit0 = sh.unit0;
        load_group(p, w);
    }
    const uint32_t tmem = sh.tmem_base;

    if (warp == 11) {
        own_plan(p, sh.own, lane);
        __syncwarp();
        if (lane == 0)
            mbar_arrive(&sh.own.ready);
        return;
    }
    if (warp == 0) {
        // ================================================================ producer
        if (lane == 0) {
            const uint64_t pol_first = policy_evict_first(), pol_keep = policy_evict_last();
            bool ok = true;
            RingPos rp{0, 0};
            int fills = 0;
            int sc = 0;
            while (ok && next_seg(p, w)) {
                const int nq = w.split() ? 1 : 2;
                if (!mbar_wait_sleep(&sh.q_empty, (sc & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&sh.q_full, nq * kQBytes);
                const int tok0 = w.seq0 * p.d.T + w.pair * (2 * kBM / p.d.G);
                for (int t = 0; t < nq; ++t)
                    for (int hf = 0; hf < 2; ++hf)
                        tma_load_3d(sh.q[t] + hf * kQHalf, &tmQ, &sh.q_full, hf * 64, w.h * p.d.G,
                                    tok0 + t * (kBM / p.d.G), pol_keep);
                ++sc;
                // pages that more than one unit reads stay in L2
                const uint64_t pol = w.pairs > 1 ? pol_keep : pol_first;
                const int32_t *const table = p.d.block_tables + (int64_t)w.seq0 * p.d.max_blocks;
                const int ahead = w.split() ? 4 : 2, nn = w.n1 - w.n0;
                // stages: score pages ahead, two at a time, then one a page
                const int pre = (min(ahead, nn) + 1) >> 1;
                for (int j = -pre; j < nn; ++j) {
                    const int x = j < 0 ? 2 * (j + pre) : j;             // K or V page of half 0
                    const int y = j < 0 ? 2 * (j + pre) + 1 : j + ahead;  // K page of half 1
                    const bool has_y = y < nn;
                    int blk[2] = {__ldg(table + w.n0 + x), has_y ? __ldg(table + w.n0 + y) : 0};
                    if (!mbar_wait_sleep(&sh.empty[rp.b], rp.ph ^ 1)) {
                        ok = false;
                        break;
                    }
                    uint64_t *const full = &sh.full[rp.b];
                    mbar_arrive_expect_tx(full, has_y ? 2 * kPageBytes : kPageBytes);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        if (e == 1 && !has_y)
                            break;
                        if (blk[e] < 0 || blk[e] >= p.d.num_blocks) {
                            // behind the pool's last row: zeros, which the softmax warps mask
                            set_err(p.d.dev_err, HSA_DEVERR_BAD_BLOCK);
                            blk[e] = p.d.num_blocks;
                        }
                        const CUtensorMap *const map = e == 0 && j >= 0 ? &tmV : &tmK;
                        const int32_t row = (blk[e] * p.d.Hkv + w.h) * kTileKeys;
                        tma_load_2d(sh.ring[rp.b][e], map, full, 0, row, pol);
                        tma_load_2d(sh.ring[rp.b][e] + kPageHalf, map, full, 64, row, pol);
                    }
                    rp.next();
                    ++fills;
                }
            }
            if (!ok)
                set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
            // drain: no TMA write may still be in flight when the CTA exits
            for (int s = 0; s < kRing && s < fills; ++s)
                mbar_wait_sleep(&sh.full[s], (fills - 1 - s) / kRing & 1);
            if (sc > 0)
                mbar_wait_sleep(&sh.q_full, (sc - 1) & 1);
        }
    } else if (warp == 1 || warp == 10) {
        // ================================================================ MMA issuers
        // The whole warp runs the loop and one elected lane issues, so that control flow
        // and descriptors stay uniform across the warp (an issuing branch of lane 0 alone
        // took 1.3 times as long a step, products in a loop that is not unrolled 1.4 times).
        const int t = warp == 10;
        const uint32_t id_s = idesc_bf16_f32(kBM, kTileKeys, 0, 0);
        const uint32_t id_pv = idesc_bf16_f32(kBM, kD, 0, 1);
        const uint32_t dhi = smem_desc_sw128_hi(1024);
        const uint32_t q_lo[2] = {smem_desc_sw128_lo(smem_u32(sh.q[0]), 16),
                                  smem_desc_sw128_lo(smem_u32(sh.q[1]), 16)};
        const uint32_t k_lo = smem_desc_sw128_lo(smem_u32(sh.ring[0][0]), 16);
        const uint32_t v_lo = smem_desc_sw128_lo(smem_u32(sh.ring[0][0]), kPageHalf);
        auto commit = [&](uint64_t *bar) {
            if (elect_one())
                tc_commit(bar);
        };
        // S region h = Q K^T, K in half e of stage b (k-step: 16 columns, 32 bytes of a
        // 128-byte swizzle row; 64 columns a block)
        auto issue_s = [&](uint32_t qa, int h, int b, int e) {
            const uint32_t kb = k_lo + (2 * b + e) * (kPageBytes >> 4);
            const uint32_t col = tmem + t * 128 + h * 64;
            const bool one = elect_one();
#pragma unroll
            for (int ks = 0; ks < kD / 16; ++ks) {
                const uint64_t qd = desc_join(qa + (ks >> 2) * (kQHalf >> 4) + (ks & 3) * 2, dhi);
                const uint64_t kd = desc_join(kb + (ks >> 2) * (kPageHalf >> 4) + (ks & 3) * 2, dhi);
                if (one) {
                    if (ks == 0)
                        tc_mma_ss_k<0>(col, qd, kd, id_s);
                    else
                        tc_mma_ss_k<1>(col, qd, kd, id_s);
                }
            }
            commit(&sh.s_full[t][h]);
        };
        // O (+)= P V: P in TMEM over S region h, V (MN-major) in half 0 of stage b (k-step:
        // 16 keys, 8 columns of bf16 pairs, 16 rows of V)
        auto issue_pv = [&](int h, int b, bool first) {
            const uint32_t vb = v_lo + 2 * b * (kPageBytes >> 4);
            const uint32_t o = tmem + kColO + t * 128, a = tmem + t * 128 + h * 64;
            const bool one = elect_one();
#pragma unroll
            for (int ks = 0; ks < kTileKeys / 16; ++ks) {
                const uint64_t vd = desc_join(vb + ks * (2048 >> 4), dhi);
                if (one) {
                    if (ks == 0)
                        tc_mma_ts(o, a, vd, id_pv, first ? 0u : 1u);
                    else
                        tc_mma_ts_k<1>(o, a + ks * 8, vd, id_pv);
                }
            }
            commit(&sh.pv_done[t]);
        };
        bool ok = true;
        RingPos rp{0, 0};
        int sc = 0;  // segments
        int c = 0;   // pages of this issuer so far: regions alternate
        int ns = 0;  // segments with a page of this issuer
        while (ok && next_seg(p, w)) {
            const bool split = w.split();
            const int nn = w.n1 - w.n0, ahead = split ? 4 : 2;
            const uint32_t qa = split || t == 0 ? q_lo[0] : q_lo[1];
            ok = mbar_wait_sleep(&sh.q_full, sc & 1);
            ++sc;
            const int pre = (min(ahead, nn) + 1) >> 1;
            for (int j = 0; j < pre && ok; ++j) {
                ok = mbar_wait_sleep(&sh.full[rp.b], rp.ph);
                if (!ok)
                    break;
                tc_fence_after();
                if (!split || t == 0)
                    issue_s(qa, split ? (c + j) & 1 : (c + 2 * j) & 1, rp.b, 0);
                if (2 * j + 1 < nn && (!split || t == 1))
                    issue_s(qa, split ? (c + j) & 1 : (c + 2 * j + 1) & 1, rp.b, 1);
                commit(&sh.empty[rp.b]);  // arrives at once where nothing was issued
                rp.next();
            }
            if (nn <= ahead + (split ? t : 0))
                commit(&sh.q_empty);  // none of this issuer's scores are left
            bool first = true;
            for (int j = 0; j < nn && ok; ++j) {
                const int b = rp.b;
                ok = mbar_wait_sleep(&sh.full[b], rp.ph);
                rp.next();
                if (!ok)
                    break;
                if (split && (j & 1) != t) {  // the other issuer's page
                    if (lane == 0)
                        mbar_arrive(&sh.empty[b]);
                    __syncwarp();
                    continue;
                }
                const int h = c & 1;
                if (!mbar_wait_sleep(&sh.p_full[t][h], (c >> 1) & 1) ||
                    (first && !mbar_wait_sleep(&sh.o_empty[t], (ns & 1) ^ 1))) {
                    ok = false;
                    break;
                }
                ++c;
                tc_fence_after();
                issue_pv(h, b, first);
                first = false;
                if (j + ahead < nn)
                    issue_s(qa, h, b, 1);
                commit(&sh.empty[b]);
                // this issuer's last scores of the segment
                if (j + ahead < nn && j + ahead + (split ? 2 : 1) >= nn)
                    commit(&sh.q_empty);
            }
            ns += first ? 0 : 1;
        }
        // every product and every arrival done before the CTA lets go of its memory
        commit(&sh.done[t]);
        if (ok)
            ok = mbar_wait_sleep(&sh.done[t], 0);
        if (!ok && lane == 0)
            set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
    } else {
        // ================================================================ softmax
        const int t = (warp - 2) >> 2;  // warpgroup: warps 2-5, warps 6-9
        const int wq = warp & 3;
        const int row = wq * 32 + lane;
        const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t col_o = kColO + t * 128;
        int c = 0;  // pages of this warpgroup so far
        bool ok = true;
        while (ok && next_seg(p, w)) {
            const int step = w.split() ? 2 : 1;
            const int first = w.n0 + (w.split() ? t : 0);
            const int r = w.pair * 2 * kBM + (w.split() ? 0 : t * kBM) + row;  // of the group and head
            const bool row_ok = r < w.ntok * p.d.G;
            float *const oct = reinterpret_cast<float *>(p.d.ws + p.slot_off) +
                               ((int64_t)blockIdx.x + w.unit) * kSlotFloats +
                               (t * kBM + row) / 8 * kOctFloats;
            if (first >= w.n1) {  // one page, not this warpgroup's
                if (row_ok) {
                    oct[row & 7] = -INFINITY;
                    oct[8 + (row & 7)] = 0.f;
                    for (int i = 0; i < kD / 4; ++i)
                        reinterpret_cast<float4 *>(oct + 16)[i * 8 + (row & 7)] =
                            make_float4(0.f, 0.f, 0.f, 0.f);
                }
                continue;
            }
            // a member may hold less than the shared pages; a row of no member (padding, not
            // written) sees every key, so that it takes no part in the choice below
            int hi_row = 0x7fffffff;
            if (row_ok)
                hi_row = clamp_len(__ldg(p.d.cached_len + w.seq0 + r / p.d.G / p.d.T));
            // O and l are in units of 2^m_used; m_want is the next page's m_used
            float m_used = -INFINITY, m_want = -INFINITY, l = 0.f;
            const int32_t *const table = p.d.block_tables + (int64_t)w.seq0 * p.d.max_blocks;
            int entry = __ldg(table + first);
            for (int n = first; n < w.n1; n += step, ++c) {
                const int next_entry = n + step < w.n1 ? __ldg(table + n + step) : 0;
                const int h = c & 1;
                const uint32_t col_s = t * 128 + h * 64;
                if (!mbar_wait_sleep(&sh.s_full[t][h], (c >> 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int hi = entry >= 0 && entry < p.d.num_blocks ? hi_row - n * kTileKeys : 0;
                // the whole warp, which stores to TMEM together, takes one way or the other
                const bool whole = __all_sync(0xffffffffu, hi >= kTileKeys);
                // ---- the row's 64 scores: one TMEM read, kept in registers ----------
                uint32_t r32[2][32];
                tmem_ld32(lane_addr + col_s, r32[0]);
                tmem_ld32(lane_addr + col_s + 32, r32[1]);
                tmem_wait_ld();
                // this page's PV-before test, whose answer is wanted after the exponents
                const bool pv_early = c == 0 || mbar_try_wait(&sh.pv_done[t], (c - 1) & 1);
                // a raise of the running maximum that the last page asked for
                float alpha = 1.f;
                bool resc = false;
                if (m_want != m_used) {
                    alpha = m_used == -INFINITY ? 1.f : fast_exp2(m_used - m_want);
                    resc = m_used != -INFINITY;
                    m_used = m_want;
                }
                const uint64_t sc2 = f2_make(p.d.scale_log2, p.d.scale_log2);
                uint32_t pk[2][16];  // P = 2^(s scale log2e - m) as bf16 pairs
                float sum = 0.f;
                auto exp_pair = [&](int c2, int i, uint64_t nb2, float &p0, float &p1) {
                    float x0, x1;
                    f2_split(f2_fma(f2_make(__uint_as_float(r32[c2][2 * i]),
                                            __uint_as_float(r32[c2][2 * i + 1])),
                                    sc2, nb2),
                             x0, x1);
                    p0 = fast_exp2(x0);
                    p1 = fast_exp2(x1);
                    pk[c2][i] = pack_bf16(p0, p1);
                };
                auto row_max = [&] {  // three-input maximum, four chains
                    float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                m4[e] = fmax3(m4[e], __uint_as_float(r32[c2][i + 2 * e]),
                                              __uint_as_float(r32[c2][i + 2 * e + 1]));
                    return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * p.d.scale_log2;
                };
                // The usual page -- all of its keys seen, a maximum there from pages before --
                // takes that maximum as it is, so that no exponent waits for this page's.  P may
                // then reach 2^kFar, which costs no precision (bf16's is relative, and the sum
                // and O are fp32), only headroom; a maximum more than kRescaleSlack higher is taken up with
                // the next page.
                bool done = false;
                if (whole && __all_sync(0xffffffffu, m_used != -INFINITY)) {
                    const uint64_t nb2 = f2_make(-m_used, -m_used);
                    uint64_t acc2[2] = {f2_make(0.f, 0.f), f2_make(0.f, 0.f)};
#pragma unroll
                    for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float p0, p1;
                            exp_pair(c2, i, nb2, p0, p1);
                            // (The row sum takes P before its rounding to bf16: unpacking the
                            // rounded pairs took the document from 129 to 134 us.  Over many
                            // keys the roundings average out; a row whose weight is on one key
                            // is off by that key's, 2^-8 of itself at most.)
                            acc2[i & 1] = f2_add(acc2[i & 1], f2_make(p0, p1));
                        }
                    const float mx = row_max();
                    float a0, a1;
                    f2_split(f2_add(acc2[0], acc2[1]), a0, a1);
                    sum = a0 + a1;
                    m_want = mx > m_used + kRescaleSlack ? mx : m_used;
                    done = __all_sync(0xffffffffu, mx <= m_used + kFar);
                }
                if (!done) {
                    // a segment's first page, keys that a row does not see, a leap of the scores:
                    // the maximum first; the row sum takes the rounded P that PV multiplies, so
                    // that a row of few keys gets no error proportional to |O|
#pragma unroll
                    for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (c2 * 32 + i >= hi)
                                r32[c2][i] = __float_as_uint(-INFINITY);
                    const float mx = row_max();
                    if (mx != -INFINITY && (m_used == -INFINITY || mx > m_used + kRescaleSlack)) {
                        if (m_used != -INFINITY) {
                            alpha *= fast_exp2(m_used - mx);
                            resc = true;
                        }
                        m_used = mx;
                    }
                    m_want = m_used;
                    const float base = m_used == -INFINITY ? 0.f : m_used;
                    const uint64_t nb2 = f2_make(-base, -base);
                    sum = 0.f;
#pragma unroll
                    for (int c2 = 0; c2 < 2; ++c2)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            float p0, p1;
                            exp_pair(c2, i, nb2, p0, p1);
                            sum += bf16_lo(pk[c2][i]) + bf16_hi(pk[c2][i]);
                        }
                }
                tmem_st16(lane_addr + col_s, pk[0]);
                tmem_st16(lane_addr + col_s + 16, pk[1]);
                // The previous page's PV is done before O is rescaled (and is waited for at
                // every page: a parity wait must see every phase).  The segment's first PV
                // overwrites O, so its first page rescales nothing.
                if (!__all_sync(0xffffffffu, pv_early) &&
                    !mbar_wait_sleep(&sh.pv_done[t], (c - 1) & 1)) {
                    ok = false;
                    break;
                }
                if (__any_sync(0xffffffffu, resc)) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c4 = 0; c4 < 4; ++c4) {
                        uint32_t o32[32];
                        tmem_ld32(lane_addr + col_o + c4 * 32, o32);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            o32[i] = __float_as_uint(__uint_as_float(o32[i]) * alpha);
                        tmem_st32(lane_addr + col_o + c4 * 32, o32);
                    }
                }
                l = l * alpha + sum;
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&sh.p_full[t][h]);
                entry = next_entry;
            }
            // ---- the segment's state -----------------------------------------------
            if (!ok || !mbar_wait_sleep(&sh.pv_done[t], (c - 1) & 1)) {
                ok = false;
                break;
            }
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
                    for (int i = 0; i < 32; i += 4)
                        dst[(c4 * 8 + i / 4) * 8] =
                            make_float4(__uint_as_float(o32[i]), __uint_as_float(o32[i + 1]),
                                        __uint_as_float(o32[i + 2]), __uint_as_float(o32[i + 3]));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&sh.o_empty[t]);
        }
        if (!ok)
            set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
    }

    // ---- part 2: every read of part 1's shared memory and TMEM is done ------------------
    tc_fence_before();
    named_bar_sync(1, kAttendThreads - 32);  // all but the plan's warp
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    const int ow = warp - 2;  // warps 2 .. 5 or 2 .. 9
    if (ow < 0 || ow >= kGroups * MT)
        return;
    if (mbar_wait_sleep(&sh.own.ready, 0))
        own_run<MT>(tmK32, tmV32, p, sh.own,
                    reinterpret_cast<uint8_t(*)[kDepth][kItemBytes]>(&sh.q[0][0]), ow / MT, ow % MT,
                    lane);
    else if (lane == 0)
        set_err(p.d.dev_err, HSA_DEVERR_TIMEOUT);
}

// ------------------------------------------------------------------------ merge, append

constexpr int kMergeThreads = 256;  // eight rows x 32 pieces of four dimensions
constexpr int kMergeCap = 32;       // states whose weights are kept at a time
constexpr int kMergeBatch = 8;      // states whose loads are in flight together

// Loads that read where `on` and give 0 elsewhere, and stay where they are written, so that a
// batch of them is in flight together.
__device__ __forceinline__ float4 load4_if(const float *p, bool on)
{
    float4 v;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
                 "mov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t"
                 "@q ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "l"(p), "r"((uint32_t)on)
                 : "memory");
    return v;
}

__device__ __forceinline__ float load_if(const float *p, bool on, float other)
{
    float v;
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.f32 %0, %3;\n\t"
                 "@q ld.global.cg.f32 %0, [%1];\n\t}"
                 : "=f"(v)
                 : "l"(p), "r"((uint32_t)on), "f"(other)
                 : "memory");
    return v;
}

// A row has a state for each part of its unit's pages that a CTA or a stream took.  A warp
// (eight rows, sixteen dimensions) collects its rows' m and l 32 states at a time, four lanes
// a row, turns them into weights, and reads o with the weights at hand.  Bound by the length
// of its instruction stream and the latency of its reads (0.6 us each from L2), not by their
// bytes (7 to 11 us for 8 to 26 MB of states): pointers step instead of being computed a state (that version ran 4000
// instructions a warp, 10 us), and four CTAs fit on an SM.
struct MergeRow {  // a row's states: own_n from own_s on, sh_n from sh_s on, sh_step floats apart
    const float *own_s, *sh_s;
    int32_t own_n, sh_n, sh_step, sh_row;
};

constexpr int kMergeStatic = kMergeThreads / 32 * kMergeCap * 8 * 4 + 8 * sizeof(MergeRow);

// Dynamic shared memory with which `share` merge CTAs fill an SM: 228 KB, of which each CTA has
// 1 KB taken off and its static arrays.
__host__ __device__ constexpr int merge_spread(int share)
{
    return (228 * 1024 / share - 1024 - kMergeStatic) & ~127;
}

// CTAS: on an SM.  Four have the registers to keep a batch's loads in flight; five are for
// grids of more than four an SM (48 sequences x 4 tokens: 72 us against 74, four samples 16
// against 15).
template <int CTAS>
__global__ void __launch_bounds__(kMergeThreads, CTAS) merge_kernel(const __grid_constant__ SharedParams p)
{
    __shared__ float wt_all[kMergeThreads / 32][kMergeCap][8];
    __shared__ MergeRow merge_rows[8];
    static_assert(sizeof(wt_all) + sizeof(merge_rows) == kMergeStatic, "static arrays");
    const DecodeParams &d = p.d;
    const int tid = threadIdx.x;
    float(&wt)[kMergeCap][8] = wt_all[tid >> 5];
    const int RT = d.G * d.T, Hq = d.G * d.Hkv;
    const int rows = d.B * RT;
    const int h = blockIdx.x % d.Hkv;
    const int oct_row = tid & 7, d4 = tid >> 3;
    const int r = (int)(blockIdx.x / d.Hkv) * 8 + oct_row;
    const bool on = r < rows;
    grid_launch_dependents();
    const int b = on ? r / RT : 0, rr = r - b * RT;
    // ---- where the eight rows' states are: a thread a row, for all of the CTA ---------------
    if (tid < 8) {
        MergeRow mr{};
        // inputs, final since before the attend kernel
        const int g = group_of(p, b);
        const int seq0 = __ldg(p.cu_group + g), seq1 = __ldg(p.cu_group + g + 1);
        grid_dependency_wait();
        if (on) {
            const OwnPlan *const own = reinterpret_cast<const OwnPlan *>(d.ws + p.own_plan_off);
            const SharedPlan *const plan = reinterpret_cast<const SharedPlan *>(d.ws + p.plan_off);
            const SharedGroup *const gp = &plan->group[g];
            const int oN = __ldcg(&own->N), oC = __ldcg(&own->C);
            const int before = __ldcg(&own->before[b]);
            const int next = b + 1 < d.B ? __ldcg(&own->before[b + 1]) : -1;
            const int N = __ldcg(&plan->N), C = __ldcg(&plan->C);
            const int item0 = __ldcg(&gp->item0);
            const int unit0 = __ldcg(&gp->unit0), pairs = __ldcg(&gp->pairs), pages = __ldcg(&gp->pages);
            {
                const int n = (next < 0 ? oN / d.Hkv : next) - before;
                const int s0 = before * d.Hkv + h * n;
                const int c_lo = part_of(s0, oN, oC), c_hi = part_of(s0 + n - 1, oN, oC);
                mr.own_n = c_hi - c_lo + 1;
                mr.own_s = reinterpret_cast<const float *>(d.ws + p.own_off) +
                           (int64_t)(c_lo + b * d.Hkv + h) * own_slot_floats(RT) + rr;
            }
            if (N > 0 && pages > 0) {
                const int rg = r - seq0 * RT;  // row of the group
                const int pair = rg / (2 * kBM), row = rg % (2 * kBM);
                const int un = h * pairs + pair;
                const int group_rows = (seq1 - seq0) * RT;
                const int wt = page_items(group_rows - pair * 2 * kBM);
                // the parts that hold the first items of the unit's first and last page
                const int s0 = item0 + h * head_items(pairs, pages, group_rows) + pair * 2 * pages;
                const int c_lo = part_of(s0, N, C), c_hi = part_of(s0 + (pages - 1) * wt, N, C);
                mr.sh_row = row & 7;
                mr.sh_s = reinterpret_cast<const float *>(d.ws + p.slot_off) +
                          (int64_t)(c_lo + unit0 + un) * kSlotFloats + row / 8 * kOctFloats + mr.sh_row;
                mr.sh_n = c_hi - c_lo + 1;
                mr.sh_step = kSlotFloats;
                // a unit in split mode left two states a row, 128 rows apart
                if (wt == 1) {
                    mr.sh_n *= 2;
                    mr.sh_step /= 2;
                }
            }
        }
        merge_rows[tid] = mr;
    }
    __syncthreads();
    // l and o of a state are l_at and o_at floats past its m
    const MergeRow mr = merge_rows[oct_row];
    const int own_step = own_slot_floats(RT), own_l = own_pad(RT);
    const int own_o = 2 * own_l - rr + rr * kD + 4 * d4;
    const int sh_o = 16 - mr.sh_row + (d4 * 8 + mr.sh_row) * 4;
    float M = -INFINITY, L = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // merges n states from s on, `step` floats apart, their l and o at l_at and o_at
    auto take = [&](const float *s, int step, int l_at, int o_at, int n) {
        const int n_warp = __reduce_max_sync(0xffffffffu, n);
        const float *sm = s + (d4 & 3) * step, *so = s + o_at;
        for (int base = 0; base < n_warp; base += kMergeCap) {
            float m[kMergeCap / 4], l[kMergeCap / 4];
            float M1 = M;
#pragma unroll
            for (int i = 0; i < kMergeCap / 4; ++i) {
                const bool some = base + 4 * i + (d4 & 3) < n;
                m[i] = load_if(sm, some, -INFINITY);
                l[i] = load_if(sm + l_at, some, 0.f);
                sm += 4 * step;
            }
#pragma unroll
            for (int i = 0; i < kMergeCap / 4; ++i)
                M1 = fmaxf(M1, m[i]);
            // the row's four lanes: 8 and 16 apart
            M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, 8));
            M1 = fmaxf(M1, __shfl_xor_sync(0xffffffffu, M1, 16));
            const float top = M1 == -INFINITY ? 0.f : M1;
            const float a = fast_exp2(M - top);  // M = -inf: o and L are 0
            M = M1;
            L *= a;
#pragma unroll
            for (int i = 0; i < kMergeCap / 4; ++i) {
                const float f = fast_exp2(m[i] - top);
                L += l[i] * f;
                wt[4 * i + (d4 & 3)][oct_row] = f;
            }
            __syncwarp();
            o.x *= a;
            o.y *= a;
            o.z *= a;
            o.w *= a;
            for (int c0 = base; c0 < min(base + kMergeCap, n_warp); c0 += kMergeBatch) {
                float4 x[kMergeBatch];
#pragma unroll
                for (int i = 0; i < kMergeBatch; ++i) {
                    x[i] = load4_if(so, c0 + i < n);
                    so += step;
                }
#pragma unroll
                for (int i = 0; i < kMergeBatch; ++i) {
                    const float f = wt[c0 - base + i][oct_row];
                    o.x += x[i].x * f;
                    o.y += x[i].y * f;
                    o.z += x[i].z * f;
                    o.w += x[i].w * f;
                }
            }
            __syncwarp();
        }
    };
    // the first own state as it is, its reads in flight with the first of the others'; the sum
    // is spread over the row's four lanes
    const float m0 = load_if(mr.own_s, on, -INFINITY);
    const float l0 = load_if(mr.own_s + own_l, on, 0.f);
    o = load4_if(mr.own_s + own_o, on);
    M = m0;
    L = (d4 & 3) == 0 ? l0 : 0.f;
    take(mr.sh_s, mr.sh_step, 8, sh_o, mr.sh_n);
    take(mr.own_s + own_step, own_step, own_l, own_o, mr.own_n - 1);
    L += __shfl_xor_sync(0xffffffffu, L, 8);
    L += __shfl_xor_sync(0xffffffffu, L, 16);
    if (on) {
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int t = rr / d.G, hh = rr % d.G;
        *reinterpret_cast<uint2 *>(d.out + ((int64_t)(b * d.T + t) * Hq + h * d.G + hh) * kD + 4 * d4) =
            make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    }
    if (d.flags & kDecodeAppend) {
        // (behind the barrier, so behind the wait: every read of the pool is done) the new rows,
        // one 16-byte chunk of K and V a thread; the grid has threads enough for all
        constexpr int kChunks = kD / 8;
        const int th = (int)blockIdx.x * (kMergeThreads / kChunks) + tid / kChunks, ch = tid % kChunks;
        if (th >= d.B * d.T * d.Hkv)
            return;
        const int bt = th / d.Hkv, hk = th - bt * d.Hkv, sb = bt / d.T;
        const int64_t pos = (int64_t)clamp_len(__ldg(d.cached_len + sb)) + bt % d.T;
        int blk = 0;
        if (pos / kTileKeys >= d.max_blocks) {
            set_err(d.dev_err, HSA_DEVERR_BAD_PAGE);
        } else if (!page_ok(p, sb, (int)(pos / kTileKeys), &blk)) {
            set_err(d.dev_err, HSA_DEVERR_BAD_BLOCK);
        } else {
            const int64_t from = (int64_t)th * kChunks + ch;
            const int64_t to = (((int64_t)blk * d.Hkv + hk) * kTileKeys + pos % kTileKeys) * kChunks + ch;
            d.k_dst[to] = __ldg(reinterpret_cast<const uint4 *>(d.k_new) + from);
            d.v_dst[to] = __ldg(reinterpret_cast<const uint4 *>(d.v_new) + from);
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
    // CTA + unit; units of part 1: 256 rows of a group and a KV head
    const size_t units = ((size_t)B * T * G / (2 * kBM) + (n_groups < B ? n_groups : B)) * Hkv;
    l.own = l.slots + pad256((ctas + units) * kSlotFloats * sizeof(float));
    l.total = l.own + ((size_t)ctas * kGroups + (size_t)B * Hkv) * own_slot_floats(G * T) * sizeof(float);
    return l;
}

bool shared_fits(const SharedParams &p)
{
    const DecodeParams &d = p.d;
    const int64_t groups = p.n_groups < d.B ? p.n_groups : d.B;
    const int64_t units = (int64_t)d.B * d.T * d.G / (2 * kBM) + groups;
    const int64_t own = kUnitCost + ((int64_t)d.max_blocks + 1) * (kTileKeys / kKT) + d.T;
    return units * 2 * d.max_blocks * d.Hkv < (int64_t)1 << 31 && own * d.B * d.Hkv < (int64_t)1 << 31 &&
           (int64_t)d.B * d.T * d.G * d.Hkv < (int64_t)1 << 30;
}

cudaError_t launch_shared(const CUtensorMap &tmK, const CUtensorMap &tmV, const CUtensorMap &tmQ,
                          const CUtensorMap &tmK32, const CUtensorMap &tmV32,
                          const SharedParams &p, int ctas, int sms, cudaStream_t stream)
{
    const size_t smem = sizeof(AttendSmem) + 1024;
    const int MT = (p.d.G * p.d.T + 15) / 16;
    auto attend = MT == 1 ? attend_kernel<1> : attend_kernel<2>;
    static SmemOptIn attend_opt[2], merge_opt;
    cudaError_t e = attend_opt[MT - 1].set(attend, smem);
    if (e == cudaSuccess)
        e = merge_opt.set(merge_kernel<4>, (size_t)merge_spread(1));
    if (e != cudaSuccess)
        return e;
    e = launch_dependent(attend, (unsigned)ctas, kAttendThreads, smem, stream, tmK,
                                           tmV, tmQ, tmK32, tmV32, p);
    if (e != cudaSuccess)
        return e;
    // Merge CTAs start while attend CTAs still hold most SMs, and would pile up on the first
    // ones to come free, whose 64 bytes a cycle then bound them (128 CTAs, 40 states a row:
    // 11 us on a quarter of the SMs, 5 us spread).  Shared memory that they do not use keeps
    // an SM to its share of the grid.
    const int64_t grid = ((int64_t)p.d.B * p.d.G * p.d.T + 7) / 8 * p.d.Hkv;
    const int64_t share = (grid + sms - 1) / sms;
    if (share > 4)
        return launch_dependent(merge_kernel<5>, (unsigned)grid, kMergeThreads, 0, stream, p);
    return launch_dependent(merge_kernel<4>, (unsigned)grid, kMergeThreads,
                            (size_t)merge_spread((int)share), stream, p);
}

}  // namespace hsa
